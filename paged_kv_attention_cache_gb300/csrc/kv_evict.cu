// Eviction from the cache by accumulated attention weight: which keys of each
// (sequence, KV head) stay, and the in-place move of their rows to the front
// of the sequence's pages.  The weights come from tl_paged_attn_decode_mass.
#include <algorithm>

#include "common.cuh"
#include "row_select.cuh"

namespace tl {

// ------------------------------------------------------------------ select --

struct EvictParams {
  const float* mass;  // [B][h_kv][mass_len]
  const int32_t* context_lens;
  int32_t* keep;      // [B][h_kv][n]
  int32_t* new_lens;  // [B]
  int64_t mass_len;
  int32_t h_kv, n, first, last;
  uint32_t* error_word;
};

template <int T>
__global__ void __launch_bounds__(T) evict_select_kernel(EvictParams P, int csize, int key_cap) {
  __shared__ SelectShared sh;
  extern __shared__ __align__(16) uint32_t sel_keys[];
  const int row = blockIdx.x / csize, rank = blockIdx.x % csize;
  const int b = row / P.h_kv;
  const int L = P.context_lens[b];
  const int len = L <= 0 || L > P.mass_len ? 0 : L;
  if (row % P.h_kv == 0 && rank == 0 && threadIdx.x == 0) {
    P.new_lens[b] = min(len, P.n);
    if (len == 0 && L > 0) report(P.error_word, TL_DEVERR_CONTEXT_RANGE);
  }
  const float* x = P.mass + (size_t)row * P.mass_len;
  int32_t* to = P.keep + (size_t)row * P.n;
  select_row<T>(
      sh, sel_keys, key_cap, x, len, P.n, P.first, P.last, rank, csize,
      [&](int pos, int i) { to[pos] = i; }, [&](int pos) { to[pos] = -1; });
}

// ----------------------------------------------------------------- compact --
//
// new row j of a (sequence, KV head) = its old row keep[j], for j < new_len,
// in place: position j and position keep[j] are slots of the same pages.  A
// CTA owns one slice of the rows (all rows, some of their bytes) of one
// (sequence, KV head) and pool, and walks j upwards in batches: it loads a
// batch's rows, and after a barrier stores them.  Every keep[j] >= j, so the
// rows a batch stores (positions below the batch's end) are never sources of
// a later batch, whatever the list's order: no row is lost, no order between
// CTAs is needed, no copy of the pool is made.  The next batch's loads are
// issued before the barrier that the current batch's stores follow, so a
// batch of reads is always in flight.  Rows that stay (keep[j] = j) are
// neither read nor written.
constexpr int kCompactThreads = 256;
constexpr int kCompactUnroll = 4;  // 16-byte vectors in flight per thread

struct CompactParams {
  void* pool[2];    // k, v: [num_pages][page_size][h_kv][row_bytes]
  float* scale[2];  // int8 pools: [num_pages][h_kv][page_size]
  float* mass;      // null, or [B][h_kv][mass_len]
  const int32_t* block_table;
  const int32_t* context_lens;
  const int32_t* keep;  // [B][h_kv][n]
  const int32_t* new_lens;
  int64_t mass_len;
  int32_t max_pages_per_seq, h_kv, num_pages, page_size, ps_shift, n;
  int32_t row_vecs, slices;  // 16-byte vectors of a row, CTAs that share a row
  uint32_t* error_word;
};

// The slot of a sequence's position j, or -1 when its page is not one.
TL_DEVINLINE int compact_slot(const CompactParams& P, const int32_t* table, int j) {
  const int blk = P.ps_shift >= 0 ? j >> P.ps_shift : j / P.page_size;
  const int page = __ldg(table + blk);
  if (page < 0 || page >= P.num_pages) return -1;
  return page * P.page_size + (j - blk * P.page_size);
}

__global__ void __launch_bounds__(kCompactThreads) compact_kernel(CompactParams P) {
  constexpr int U = kCompactUnroll;
  const int tid = threadIdx.x;
  const int row = blockIdx.x, b = row / P.h_kv, g = row % P.h_kv;
  const int L = P.context_lens[b], new_len = P.new_lens[b];
  const int64_t cap = (int64_t)P.max_pages_per_seq * P.page_size;
  const bool bad_len = L > cap || (P.mass && L > P.mass_len) || new_len < 0 || new_len > P.n ||
                       new_len > max(L, 0);
  if (bad_len) {  // the sequence stays as it is
    if (blockIdx.y == 0 && tid == 0) report(P.error_word, TL_DEVERR_CONTEXT_RANGE);
    return;
  }
  const int32_t* keep = P.keep + (size_t)row * P.n;
  const int32_t* table = P.block_table + (size_t)b * P.max_pages_per_seq;
  if ((int)blockIdx.y == 2 * P.slices) {  // the masses move with their keys
    float* m = P.mass + (size_t)row * P.mass_len;
    for (int j0 = 0; j0 < new_len; j0 += kCompactThreads * U) {
      float v[U];
      bool mv[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int j = j0 + u * kCompactThreads + tid;
        const int s = j < new_len ? __ldg(keep + j) : 0;
        mv[u] = j < new_len && s > j && s < L;
        v[u] = mv[u] ? __ldcg(m + s) : 0.f;
      }
      __syncthreads();
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (mv[u]) m[j0 + u * kCompactThreads + tid] = v[u];
    }
    // positions that no key holds any more gather nothing: the last batch's
    // loads are behind a barrier, so they may be cleared
    __syncthreads();
    for (int j = new_len + tid; j < L; j += kCompactThreads) m[j] = 0.f;
    return;
  }
  const int which = blockIdx.y / P.slices, slice = blockIdx.y % P.slices;
  const int lanes = P.row_vecs / P.slices;  // threads of a row
  const int per = kCompactThreads / lanes;  // rows of a pass
  const int r = tid / lanes, c = slice * lanes + tid % lanes;
  const bool active = r < per;
  uint4* pool = static_cast<uint4*>(which ? P.pool[1] : P.pool[0]);
  float* scale = which ? P.scale[1] : P.scale[0];
  const bool moves_scale = scale && slice == 0 && tid % lanes == 0;
  const int batch = per * U;
  uint4 v[U], nv[U];
  float sv[U], nsv[U];
  int dst[U], ndst[U];  // the row's slot, -1: nothing to store
  auto load = [&](int j0, uint4* x, float* sx, int* d) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int j = j0 + u * per + r;
      d[u] = -1;
      if (!active || j >= new_len) continue;
      const int s = __ldg(keep + j);
      if (s == j) continue;
      if (s < j || s >= L) {
        if (tid % lanes == 0) report(P.error_word, TL_DEVERR_CONTEXT_RANGE);
        continue;
      }
      const int from = compact_slot(P, table, s), to = compact_slot(P, table, j);
      if (from < 0 || to < 0) {
        if (tid % lanes == 0) report(P.error_word, TL_DEVERR_PAGE_RANGE);
        continue;
      }
      d[u] = to;
      x[u] = __ldcg(pool + ((size_t)from * P.h_kv + g) * P.row_vecs + c);
      if (moves_scale)
        sx[u] = __ldcg(scale + ((size_t)(from / P.page_size) * P.h_kv + g) * P.page_size +
                       from % P.page_size);
    }
  };
  load(0, v, sv, dst);
  for (int j0 = 0; j0 < new_len; j0 += batch) {
    load(j0 + batch, nv, nsv, ndst);
    __syncthreads();  // every thread's loads of this batch come before any store of it
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (dst[u] >= 0) {
        pool[((size_t)dst[u] * P.h_kv + g) * P.row_vecs + c] = v[u];
        if (moves_scale)
          scale[((size_t)(dst[u] / P.page_size) * P.h_kv + g) * P.page_size +
                dst[u] % P.page_size] = sv[u];
      }
      v[u] = nv[u];
      sv[u] = nsv[u];
      dst[u] = ndst[u];
    }
  }
}

static tl_status compact_impl(void* k, void* v, float* k_scales, float* v_scales,
                              const int32_t* block_table, int32_t max_pages_per_seq,
                              const int32_t* context_lens, const int32_t* keep, int32_t n_keep,
                              const int32_t* new_lens, float* mass, int32_t mass_len, int32_t B,
                              int32_t h_kv, int32_t d, int32_t num_pages, int32_t page_size,
                              int elem, uint32_t* error_word, void* stream) {
  if (B <= 0 || h_kv <= 0 || d <= 0 || num_pages <= 0 || page_size <= 0 ||
      max_pages_per_seq <= 0 || n_keep <= 0 || (mass && mass_len <= 0))
    return TL_ERR_INVALID_ARG;
  if (!k || !v || !block_table || !context_lens || !keep || !new_lens) return TL_ERR_INVALID_ARG;
  if (!aligned16(k) || !aligned16(v) || !aligned16(k_scales) || !aligned16(v_scales) ||
      !aligned16(keep) || !aligned16(new_lens) || !aligned16(mass) ||
      (reinterpret_cast<uintptr_t>(block_table) & 3u) ||
      (reinterpret_cast<uintptr_t>(context_lens) & 3u))
    return TL_ERR_INVALID_ARG;
  if (elem == 0) return TL_ERR_UNSUPPORTED;
  const int64_t row_bytes = (int64_t)d * elem;
  if (row_bytes % 16 != 0) return TL_ERR_INVALID_ARG;
  if (row_bytes / 16 > kCompactThreads || page_size > 256 ||
      (int64_t)num_pages * page_size >= ((int64_t)1 << 31) || (int64_t)B * h_kv > INT32_MAX)
    return TL_ERR_UNSUPPORTED;
  CompactParams P;
  P.pool[0] = k;
  P.pool[1] = v;
  P.scale[0] = k_scales;
  P.scale[1] = v_scales;
  P.mass = mass;
  P.block_table = block_table;
  P.context_lens = context_lens;
  P.keep = keep;
  P.new_lens = new_lens;
  P.mass_len = mass_len;
  P.max_pages_per_seq = max_pages_per_seq;
  P.h_kv = h_kv;
  P.num_pages = num_pages;
  P.page_size = page_size;
  P.ps_shift = -1;
  for (int s = 0; s < 9; ++s)
    if ((1 << s) == page_size) P.ps_shift = s;
  P.n = n_keep;
  P.row_vecs = (int32_t)(row_bytes / 16);
  P.error_word = error_word;
  // a row is shared by more CTAs while the (sequence, head) rows leave SMs
  // empty, down to 64 bytes of a row
  const int64_t rows = (int64_t)B * h_kv;
  P.slices = 1;
  while (P.row_vecs % (2 * P.slices) == 0 && P.row_vecs / (2 * P.slices) >= 4 &&
         rows * 2 * P.slices < 2 * num_sms())
    P.slices *= 2;
  const dim3 grid((unsigned)rows, (unsigned)(2 * P.slices + (mass ? 1 : 0)));
  compact_kernel<<<grid, kCompactThreads, 0, (cudaStream_t)stream>>>(P);
  return launch_status();
}

}  // namespace tl

// -------------------------------------------------------------------- host --

extern "C" tl_status tl_kv_evict_select(const float* mass, int32_t mass_len,
                                        const int32_t* context_lens, int32_t n_keep,
                                        int32_t keep_first, int32_t keep_last, int32_t* keep,
                                        int32_t* new_lens, int32_t B, int32_t h_kv,
                                        uint32_t* error_word, void* stream) {
  using namespace tl;
  if (B <= 0 || h_kv <= 0 || mass_len <= 0 || n_keep <= 0 || keep_first < 0 || keep_last < 0 ||
      (int64_t)keep_first + keep_last > n_keep)
    return TL_ERR_INVALID_ARG;
  if (!mass || !context_lens || !keep || !new_lens) return TL_ERR_INVALID_ARG;
  if (!aligned16(mass) || !aligned16(keep) || !aligned16(new_lens) ||
      (reinterpret_cast<uintptr_t>(context_lens) & 3u))
    return TL_ERR_INVALID_ARG;
  if ((int64_t)B * h_kv > INT32_MAX / 8 || mass_len > (1 << 30) || n_keep > (1 << 30))
    return TL_ERR_UNSUPPORTED;
  EvictParams P;
  P.mass = mass;
  P.context_lens = context_lens;
  P.keep = keep;
  P.new_lens = new_lens;
  P.mass_len = mass_len;
  P.h_kv = h_kv;
  P.n = n_keep;
  P.first = keep_first;
  P.last = keep_last;
  P.error_word = error_word;
  const int64_t rows = (int64_t)B * h_kv;
  const SelectShape s = select_shape(rows, mass_len);
  int csize = s.cluster, key_cap = s.keys;
  void* args[] = {&P, &csize, &key_cap};
  const void* const kernels[3] = {reinterpret_cast<const void*>(evict_select_kernel<256>),
                                  reinterpret_cast<const void*>(evict_select_kernel<512>),
                                  reinterpret_cast<const void*>(evict_select_kernel<1024>)};
  if (launch_rows(kernels, rows, s, args, false, (cudaStream_t)stream) != cudaSuccess)
    return TL_ERR_CUDA;
  return launch_status();
}

extern "C" tl_status tl_kv_cache_compact(void* k_cache, void* v_cache, const int32_t* block_table,
                                         int32_t max_pages_per_seq, const int32_t* context_lens,
                                         const int32_t* keep, int32_t n_keep,
                                         const int32_t* new_lens, float* mass, int32_t mass_len,
                                         int32_t B, int32_t h_kv, int32_t d, int32_t num_pages,
                                         int32_t page_size, tl_dtype dtype, uint32_t* error_word,
                                         void* stream) {
  const int elem = dtype == TL_F32 ? 4 : dtype == TL_BF16 ? 2 : dtype == TL_FP8_E4M3 ? 1 : 0;
  return tl::compact_impl(k_cache, v_cache, nullptr, nullptr, block_table, max_pages_per_seq,
                          context_lens, keep, n_keep, new_lens, mass, mass_len, B, h_kv, d,
                          num_pages, page_size, elem, error_word, stream);
}

extern "C" tl_status tl_kv_cache_compact_int8(int8_t* k_codes, int8_t* v_codes, float* k_scales,
                                              float* v_scales, const int32_t* block_table,
                                              int32_t max_pages_per_seq,
                                              const int32_t* context_lens, const int32_t* keep,
                                              int32_t n_keep, const int32_t* new_lens, float* mass,
                                              int32_t mass_len, int32_t B, int32_t h_kv, int32_t d,
                                              int32_t num_pages, int32_t page_size,
                                              uint32_t* error_word, void* stream) {
  if (!k_scales || !v_scales) return TL_ERR_INVALID_ARG;
  return tl::compact_impl(k_codes, v_codes, k_scales, v_scales, block_table, max_pages_per_seq,
                          context_lens, keep, n_keep, new_lens, mass, mass_len, B, h_kv, d,
                          num_pages, page_size, 1, error_word, stream);
}
