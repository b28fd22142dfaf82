// Eviction from the cache by accumulated attention weight: which keys of each
// (sequence, KV head) stay, and the in-place move of their rows to the front
// of the sequence's pages.  The weights come from tl_paged_attn_decode_mass.
// (Eviction by accumulated weight with the newest keys protected: Zhang et al.,
// "H2O: Heavy-Hitter Oracle for Efficient Generative Inference of Large Language
// Models", 2023.)
#include <algorithm>

#include "common.cuh"
#include "rope.cuh"
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

template <int T, bool FITS>
__global__ void __launch_bounds__(T) evict_select_kernel(EvictParams P, int csize, int key_cap) {
  __shared__ SelectShared<T> sh;
  extern __shared__ __align__(16) uint32_t sel_keys[];
  const int row = (int)blockIdx.x >> (31 - __clz(csize)), rank = (int)blockIdx.x & (csize - 1);
  const int b = row / P.h_kv;
  const int L = P.context_lens[b];
  const int len = L <= 0 || L > P.mass_len ? 0 : L;
  if (row % P.h_kv == 0 && rank == 0 && threadIdx.x == 0) {
    P.new_lens[b] = min(len, P.n);
    if (len == 0 && L > 0) report(P.error_word, TL_DEVERR_CONTEXT_RANGE);
  }
  const float* x = P.mass + (size_t)row * P.mass_len;
  int32_t* to = P.keep + (size_t)row * P.n;
  select_row<T, FITS>(
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
// CTAs is needed, no copy of the pool is made.  Reads may run ahead of the
// stores as far as registers go: a batch's list entries are loaded two
// batches ahead and its rows one batch ahead, before the barrier that the
// stores of the batch before them follow.  Rows that stay (keep[j] = j) are
// neither read nor written.  Bound: HBM, 2 x (K and V row) per moved row.
// Measured (bf16, 8 KV heads of 128): 64 sequences of 512-8,192 keys cut to
// 2,048 in 151 us (871 MB at 5.8 TB/s), one of 32,768 cut to 8,192 in 23 us (69
// MB, 3.0 TB/s: its CTAs wait for a batch's loads, 8 batches in a row, and a
// row's 32-byte pieces fill the L1's tag rate by half).  Copies through a ring
// in shared memory, two and more batches ahead of the stores, were slower
// (165-190 and 25-27 us).
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

// Page and offset of a sequence's position j; page -1 when it is not one of
// the pool's.
struct CompactPlace {
  int page, off;
};
TL_DEVINLINE CompactPlace compact_place(const CompactParams& P, const int32_t* table, int j) {
  const int blk = P.ps_shift >= 0 ? j >> P.ps_shift : j / P.page_size;
  const int page = __ldg(table + blk);
  return {page >= 0 && page < P.num_pages ? page : -1, j - blk * P.page_size};
}

// The walk: rows_per_pass rows of a pass, this thread's being row r of it
// (r < 0: none), U passes a batch.  slot(j): where position j's element is
// (-1: nowhere); get(slot): the element; put(slot, x, by): its new place, `by`
// positions from the old one (put of every element, moved or not, in step with
// the warp's other threads, where ALL).  Entries outside [j, L) and positions
// without a page are reported by `reports` threads and skipped.
template <int U, class Vec, class Index, bool ALL, class Slot, class Get, class Put>
TL_DEVINLINE void compact_walk(const int32_t* keep, int new_len, int L, int rows_per_pass, int r,
                               bool reports, uint32_t* error_word, Slot slot, Get get, Put put) {
  const int batch = rows_per_pass * U;
  auto entry = [&](int j) { return r >= 0 && j < new_len ? __ldg(keep + j) : j; };
  // the rows of the batch at j0, whose list entries are s
  auto load = [&](int j0, const int* s, Vec* x, Index* d, int* by) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int j = j0 + u * rows_per_pass + r;
      d[u] = -1;
      if (s[u] == j) continue;  // stays, or not a row of this thread
      if (s[u] < j || s[u] >= L) {
        if (reports) report(error_word, TL_DEVERR_CONTEXT_RANGE);
        continue;
      }
      const Index from = slot(s[u]), to = slot(j);
      if (from < 0 || to < 0) {
        if (reports) report(error_word, TL_DEVERR_PAGE_RANGE);
        continue;
      }
      d[u] = to;
      by[u] = j - s[u];
      x[u] = get(from);
    }
  };
  Vec v[U], nv[U];
  Index dst[U], ndst[U];
  int s[U], ns[U], by[U], nby[U];
#pragma unroll
  for (int u = 0; u < U; ++u) s[u] = entry(u * rows_per_pass + r);
#pragma unroll
  for (int u = 0; u < U; ++u) ns[u] = entry(batch + u * rows_per_pass + r);
  load(0, s, v, dst, by);
  for (int j0 = 0; j0 < new_len; j0 += batch) {
#pragma unroll
    for (int u = 0; u < U; ++u) s[u] = entry(j0 + 2 * batch + u * rows_per_pass + r);
    load(j0 + batch, ns, nv, ndst, nby);
    __syncthreads();  // every thread's loads of this batch come before any store of it
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (ALL || dst[u] >= 0) put(dst[u], v[u], by[u]);
      v[u] = nv[u];
      dst[u] = ndst[u];
      by[u] = nby[u];
      ns[u] = s[u];
    }
  }
}

// A sequence's lengths, checked; false: it stays as it is.
TL_DEVINLINE bool compact_lens(const CompactParams& P, int b, int& L, int& new_len) {
  L = P.context_lens[b];
  new_len = P.new_lens[b];
  const int64_t cap = (int64_t)P.max_pages_per_seq * P.page_size;
  const bool bad = L > cap || (P.mass && L > P.mass_len) || new_len < 0 || new_len > P.n ||
                   new_len > max(L, 0);
  if (bad && blockIdx.y == 0 && threadIdx.x == 0) report(P.error_word, TL_DEVERR_CONTEXT_RANGE);
  return !bad;
}

// Rows as they are: this CTA's slice (of `slices`) of one pool's rows.
template <int T, int U>
TL_DEVINLINE void compact_rows(const CompactParams& P, void* rows, int slices, int slice, int g,
                               const int32_t* keep, const int32_t* table, int L, int new_len) {
  const int tid = threadIdx.x;
  const int lanes = P.row_vecs / slices;  // threads of a row
  const int per = T / lanes;              // rows of a pass
  uint4* pool =
      static_cast<uint4*>(rows) + (size_t)g * P.row_vecs + slice * lanes + tid % lanes;
  const int64_t stride = (int64_t)P.h_kv * P.row_vecs;
  compact_walk<U, uint4, int, false>(
      keep, new_len, L, per, tid / lanes < per ? tid / lanes : -1, tid % lanes == 0,
      P.error_word,
      [&](int j) {
        const CompactPlace p = compact_place(P, table, j);
        return p.page < 0 ? -1 : p.page * P.page_size + p.off;
      },
      [&](int slot) { return __ldcg(pool + slot * stride); },
      [&](int slot, const uint4& x, int) { pool[slot * stride] = x; });
}

// The scales of an int8 pool's rows.
template <int T, int U>
TL_DEVINLINE void compact_scales(const CompactParams& P, float* scales, int g,
                                 const int32_t* keep, const int32_t* table, int L, int new_len) {
  float* scale = scales + (size_t)g * P.page_size;
  compact_walk<U, float, int64_t, false>(
      keep, new_len, L, T, threadIdx.x, false, nullptr,
      [&](int j) -> int64_t {
        const CompactPlace p = compact_place(P, table, j);
        return p.page < 0 ? -1 : (int64_t)p.page * P.h_kv * P.page_size + p.off;
      },
      [&](int64_t slot) { return __ldcg(scale + slot); },
      [&](int64_t slot, float x, int) { scale[slot] = x; });
}

template <int T, int U>
TL_DEVINLINE void compact_mass(const CompactParams& P, int row, const int32_t* keep, int L,
                               int new_len) {
  float* m = P.mass + (size_t)row * P.mass_len;
  compact_walk<U, float, int, false>(
      keep, new_len, L, T, threadIdx.x, false, nullptr, [&](int j) { return j; },
      [&](int j) { return __ldcg(m + j); }, [&](int j, float x, int) { m[j] = x; });
  // positions that no key holds any more gather nothing; the last batch's
  // loads are behind the walk's barrier
  __syncthreads();
  for (int j = new_len + (int)threadIdx.x; j < L; j += T) m[j] = 0.f;
}

template <int T, int U>
__global__ void __launch_bounds__(T) compact_kernel(CompactParams P) {
  const int row = blockIdx.x, b = row / P.h_kv, g = row % P.h_kv;
  int L, new_len;
  if (!compact_lens(P, b, L, new_len)) return;
  const int32_t* keep = P.keep + (size_t)row * P.n;
  const int32_t* table = P.block_table + (size_t)b * P.max_pages_per_seq;
  const int kind = blockIdx.y;  // the pools' slices, then K and V scales, then the mass
  if (kind < 2 * P.slices) {
    const bool is_v = kind >= P.slices;
    compact_rows<T, U>(P, is_v ? P.pool[1] : P.pool[0], P.slices, kind - (is_v ? P.slices : 0), g,
                       keep, table, L, new_len);
  } else if (P.scale[0] && kind < 2 * P.slices + 2) {
    compact_scales<T, U>(P, kind == 2 * P.slices ? P.scale[0] : P.scale[1], g, keep, table, L,
                         new_len);
  } else {
    compact_mass<T, U>(P, row, keep, L, new_len);
  }
}

// The same with K rows turned by the positions they move (tl_kv_cache_compact_rope).
// K rows are walked in rotary units (rope.cuh), one a thread, which turns its 8
// pairs between the load and the store: a row that moves has an angle of its
// own for every pair.  int8 rows are scaled anew over their threads, which lie
// in one warp (d is a power of two up to 512).
struct CompactTurn {
  const uint64_t* freqs;
  int32_t rot, interleaved;
  int32_t units, slices;  // rotary units of a row, CTAs that share a K row
};

template <int E>
struct CompactUnit : RopeUnit<E, E == kElemF32 ? 4 : 8> {
  float scale;  // int8
};

template <int T, int U, int E, bool INTER>
__global__ void __launch_bounds__(T) compact_rope_kernel(CompactParams P, CompactTurn R) {
  const int tid = threadIdx.x;
  const int row = blockIdx.x, b = row / P.h_kv, g = row % P.h_kv;
  int L, new_len;
  if (!compact_lens(P, b, L, new_len)) return;
  const int32_t* keep = P.keep + (size_t)row * P.n;
  const int32_t* table = P.block_table + (size_t)b * P.max_pages_per_seq;
  const int kind = blockIdx.y;  // K slices, V slices, V scales (int8), the mass
  if (kind < R.slices) {
    const int lanes = R.units / R.slices, per = T / lanes;
    const int u = kind * lanes + tid % lanes;
    constexpr int W = 16 / CompactUnit<E>::NW;
    using Pairs = RopePairs<INTER, W>;
    int at[16 / W];
    rope_unit_words<INTER, W>(u, R.units * 16, R.rot, at);
    const int64_t row_bytes = (int64_t)P.row_vecs * 16, stride = P.h_kv * row_bytes;
    char* pool = static_cast<char*>(P.pool[0]) + g * row_bytes;
    float* scales = E == kElemInt8 ? P.scale[0] + (size_t)g * P.page_size : nullptr;
    auto scale_at = [&](int slot) {
      const int page = P.ps_shift >= 0 ? slot >> P.ps_shift : slot / P.page_size;
      return scales + (int64_t)page * (P.h_kv - 1) * P.page_size + slot;
    };
    compact_walk<U, CompactUnit<E>, int, E == kElemInt8>(
        keep, new_len, L, per, tid / lanes < per ? tid / lanes : -1, tid % lanes == 0,
        P.error_word,
        [&](int j) {
          const CompactPlace p = compact_place(P, table, j);
          return p.page < 0 ? -1 : p.page * P.page_size + p.off;
        },
        [&](int slot) {
          CompactUnit<E> x;
          x.load(pool + slot * stride, at);
          if constexpr (E == kElemInt8) x.scale = __ldcg(scale_at(slot));
          return x;
        },
        [&](int slot, CompactUnit<E>& x, int by) {
          float y[16];
          if (E != kElemInt8 && (INTER ? at[0] >= R.rot : 16 * u >= R.rot)) {
            x.store(pool + slot * stride, at);
            return;
          }
          x.values(y);
          if constexpr (E == kElemInt8) {
#pragma unroll
            for (int k = 0; k < 16; ++k) y[k] *= x.scale;
          }
          if (slot >= 0)
            rope_unit_rotate<INTER, W>(
                y, [&](int k) { return Pairs::turn(at, k, u, R.rot); },
                [&](int k) { return rope_turn(__ldg(R.freqs + Pairs::index(at, k)), by); });
          if constexpr (E == kElemInt8) {
            bool bad = false;
            float m = rope_unit_max(y, bad);
            for (int o = lanes >> 1; o > 0; o >>= 1)
              m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
            if (slot < 0) return;
            const float sc = __fdiv_rn(m, 127.f);
            x.set_codes(y, sc, !bad);
            if (tid % lanes == 0) *scale_at(slot) = sc;
            if (bad) report(P.error_word, TL_DEVERR_VALUE_RANGE);
          } else {
            const CompactUnit<E> was = x;
            x.set(y);
            if (INTER) {  // words behind the rotated part keep their bits
#pragma unroll
              for (int w = 0; w < x.NW; ++w)
                if (at[w] >= R.rot) x.w[w] = was.w[w];
            }
          }
          x.store(pool + slot * stride, at);
        });
  } else if (kind < R.slices + P.slices) {
    compact_rows<T, U>(P, P.pool[1], P.slices, kind - R.slices, g, keep, table, L, new_len);
  } else if (E == kElemInt8 && kind == R.slices + P.slices) {
    compact_scales<T, U>(P, P.scale[1], g, keep, table, L, new_len);
  } else {
    compact_mass<T, U>(P, row, keep, L, new_len);
  }
}

static tl_status compact_impl(void* k, void* v, float* k_scales, float* v_scales,
                              const int32_t* block_table, int32_t max_pages_per_seq,
                              const int32_t* context_lens, const int32_t* keep, int32_t n_keep,
                              const int32_t* new_lens, float* mass, int32_t mass_len, int32_t B,
                              int32_t h_kv, int32_t d, int32_t num_pages, int32_t page_size,
                              int elem, uint32_t* error_word, void* stream,
                              CompactTurn* turn = nullptr) {
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
  if (turn) {
    if (turn->rot < 2 || turn->rot % 2 || turn->rot > d || !turn->freqs ||
        (reinterpret_cast<uintptr_t>(turn->freqs) & 7u))
      return TL_ERR_INVALID_ARG;
    if (d % 16 || turn->rot % 16 || (k_scales && ((d & (d - 1)) || d > 512)))
      return TL_ERR_UNSUPPORTED;
  }
  if (row_bytes > 4096 || page_size > 256 ||
      (int64_t)num_pages * page_size >= ((int64_t)1 << 31) || (int64_t)B * h_kv > INT32_MAX ||
      n_keep > (1 << 30) || (mass && mass_len > (1 << 30)))
    return TL_ERR_UNSUPPORTED;
  // each pool (and the mass) is moved by CTAs of its own: one buffer given for
  // two of them would be moved twice at once
  const size_t pool_bytes = (size_t)num_pages * page_size * h_kv * row_bytes;
  const size_t scale_bytes = k_scales ? sizeof(float) * (size_t)num_pages * page_size * h_kv : 0;
  const struct {
    const void* p;
    size_t bytes;
  } moved[] = {{k, pool_bytes},
               {v, pool_bytes},
               {k_scales, scale_bytes},
               {v_scales, scale_bytes},
               {mass, mass ? sizeof(float) * (size_t)B * h_kv * mass_len : 0}};
  for (int i = 0; i < 5; ++i)
    for (int j = 0; j < i; ++j)
      if (moved[i].bytes && moved[j].bytes &&
          overlap(moved[i].p, moved[i].bytes, moved[j].p, moved[j].bytes))
        return TL_ERR_INVALID_ARG;
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
  // empty, down to 32 bytes (a sector) of a row; then a CTA takes all of an SM's threads
  const int64_t rows = (int64_t)B * h_kv;
  P.slices = 1;
  while (P.row_vecs % (2 * P.slices) == 0 && P.row_vecs / (2 * P.slices) >= 2 &&
         rows * 2 * P.slices < 2 * num_sms())
    P.slices *= 2;
  if (turn) {
    // K rows alike, a slice being units whose words fill whole 32-byte sectors
    // (an int8 row is one slice, for its scale)
    CompactTurn R = *turn;
    R.units = d / 16;
    R.slices = 1;
    const int least = elem == 1 ? 4 : 2;  // words of 8 bytes, or of 16
    if (!k_scales)
      while (R.units % (2 * R.slices) == 0 && R.units / (2 * R.slices) >= least &&
             rows * 2 * R.slices < 2 * num_sms())
        R.slices *= 2;
    const bool big = rows * 2 * P.slices <= 2 * num_sms() || P.row_vecs / P.slices > 128 ||
                     R.units / R.slices > 128;
    const dim3 grid((unsigned)rows, (unsigned)(R.slices + P.slices + (k_scales ? 1 : 0) +
                                               (mass ? 1 : 0)));
    cudaStream_t st = (cudaStream_t)stream;
#define TL_COMPACT_ROPE(E)                                          \
  do {                                                              \
    auto kern = big ? (R.interleaved ? compact_rope_kernel<512, 2, E, true>  \
                                     : compact_rope_kernel<512, 2, E, false>) \
                    : (R.interleaved ? compact_rope_kernel<128, 4, E, true>   \
                                     : compact_rope_kernel<128, 4, E, false>); \
    kern<<<grid, big ? 512 : 128, 0, st>>>(P, R);                             \
  } while (0)
    if (k_scales) TL_COMPACT_ROPE(kElemInt8);
    else if (elem == 1) TL_COMPACT_ROPE(kElemE4m3);
    else if (elem == 2) TL_COMPACT_ROPE(kElemBf16);
    else TL_COMPACT_ROPE(kElemF32);
#undef TL_COMPACT_ROPE
    return launch_status();
  }
  const dim3 grid((unsigned)rows, (unsigned)(2 * P.slices + (k_scales ? 2 : 0) + (mass ? 1 : 0)));
  // otherwise small CTAs, whose barriers hold few rows back: one sequence of
  // 8,192 rows kept takes 23 us with 1,024 threads and 33 with 512, 64
  // sequences of 2,048 take 152 us with 128 threads, 169 with 256, 212 with 64
  if (rows * 2 * P.slices <= 2 * num_sms() || P.row_vecs / P.slices > 128)
    compact_kernel<1024, 2><<<grid, 1024, 0, (cudaStream_t)stream>>>(P);
  else
    compact_kernel<128, 4><<<grid, 128, 0, (cudaStream_t)stream>>>(P);
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
  // a row's CTAs read the lengths and masses while others write: in place, a
  // head could see the length that another one's CTA has already cut
  const size_t rows_bytes = sizeof(int32_t) * (size_t)B * h_kv, lens_bytes = sizeof(int32_t) * (size_t)B;
  if (overlap(new_lens, lens_bytes, context_lens, lens_bytes) ||
      overlap(keep, rows_bytes * n_keep, context_lens, lens_bytes) ||
      overlap(keep, rows_bytes * n_keep, new_lens, lens_bytes) ||
      overlap(keep, rows_bytes * n_keep, mass, rows_bytes * mass_len) ||
      overlap(new_lens, lens_bytes, mass, rows_bytes * mass_len))
    return TL_ERR_INVALID_ARG;
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
  const void* const kernels[4] = {reinterpret_cast<const void*>(evict_select_kernel<256, true>),
                                  reinterpret_cast<const void*>(evict_select_kernel<512, true>),
                                  reinterpret_cast<const void*>(evict_select_kernel<1024, true>),
                                  reinterpret_cast<const void*>(evict_select_kernel<1024, false>)};
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

extern "C" tl_status tl_kv_cache_compact_rope(
    void* k_cache, void* v_cache, const int32_t* block_table, int32_t max_pages_per_seq,
    const int32_t* context_lens, const int32_t* keep, int32_t n_keep, const int32_t* new_lens,
    float* mass, int32_t mass_len, const uint64_t* freqs, int32_t rot_dim, int32_t interleaved,
    int32_t B, int32_t h_kv, int32_t d, int32_t num_pages, int32_t page_size, tl_dtype dtype,
    uint32_t* error_word, void* stream) {
  const int elem = dtype == TL_F32 ? 4 : dtype == TL_BF16 ? 2 : dtype == TL_FP8_E4M3 ? 1 : 0;
  tl::CompactTurn turn = {freqs, rot_dim, interleaved != 0, 0, 0};
  return tl::compact_impl(k_cache, v_cache, nullptr, nullptr, block_table, max_pages_per_seq,
                          context_lens, keep, n_keep, new_lens, mass, mass_len, B, h_kv, d,
                          num_pages, page_size, elem, error_word, stream, &turn);
}

extern "C" tl_status tl_kv_cache_compact_rope_int8(
    int8_t* k_codes, int8_t* v_codes, float* k_scales, float* v_scales,
    const int32_t* block_table, int32_t max_pages_per_seq, const int32_t* context_lens,
    const int32_t* keep, int32_t n_keep, const int32_t* new_lens, float* mass, int32_t mass_len,
    const uint64_t* freqs, int32_t rot_dim, int32_t interleaved, int32_t B, int32_t h_kv,
    int32_t d, int32_t num_pages, int32_t page_size, uint32_t* error_word, void* stream) {
  if (!k_scales || !v_scales) return TL_ERR_INVALID_ARG;
  tl::CompactTurn turn = {freqs, rot_dim, interleaved != 0, 0, 0};
  return tl::compact_impl(k_codes, v_codes, k_scales, v_scales, block_table, max_pages_per_seq,
                          context_lens, keep, n_keep, new_lens, mass, mass_len, B, h_kv, d,
                          num_pages, page_size, 1, error_word, stream, &turn);
}
