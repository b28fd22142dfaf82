// Eviction from the cache by accumulated attention weight: which keys of each
// (sequence, KV head) stay, and the in-place move of their rows to the front
// of the sequence's pages.  The weights come from tl_paged_attn_decode_mass.
// (Eviction by accumulated weight with the newest keys protected: Zhang et al.,
// "H2O: Heavy-Hitter Oracle for Efficient Generative Inference of Large Language
// Models", 2023.)
#include <algorithm>
#include <atomic>

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
// (-1: nowhere); at(slot): the element.  Entries outside [j, L) and positions
// without a page are reported by `reports` threads and skipped.
template <int U, class Vec, class Index, class Slot, class At>
TL_DEVINLINE void compact_walk(const int32_t* keep, int new_len, int L, int rows_per_pass, int r,
                               bool reports, uint32_t* error_word, Slot slot, At at) {
  const int batch = rows_per_pass * U;
  auto entry = [&](int j) { return r >= 0 && j < new_len ? __ldg(keep + j) : j; };
  // the rows of the batch at j0, whose list entries are s
  auto load = [&](int j0, const int* s, Vec* x, Index* d) {
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
      x[u] = __ldcg(at(from));
    }
  };
  Vec v[U], nv[U];
  Index dst[U], ndst[U];
  int s[U], ns[U];
#pragma unroll
  for (int u = 0; u < U; ++u) s[u] = entry(u * rows_per_pass + r);
#pragma unroll
  for (int u = 0; u < U; ++u) ns[u] = entry(batch + u * rows_per_pass + r);
  load(0, s, v, dst);
  for (int j0 = 0; j0 < new_len; j0 += batch) {
#pragma unroll
    for (int u = 0; u < U; ++u) s[u] = entry(j0 + 2 * batch + u * rows_per_pass + r);
    load(j0 + batch, ns, nv, ndst);
    __syncthreads();  // every thread's loads of this batch come before any store of it
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (dst[u] >= 0) *at(dst[u]) = v[u];
      v[u] = nv[u];
      dst[u] = ndst[u];
      ns[u] = s[u];
    }
  }
}

template <int T, int U>
__global__ void __launch_bounds__(T) compact_kernel(CompactParams P) {
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
  const int kind = blockIdx.y;  // the pools' slices, then K and V scales, then the mass
  if (kind < 2 * P.slices) {
    const bool is_v = kind >= P.slices;
    const int lanes = P.row_vecs / P.slices;  // threads of a row
    const int per = T / lanes;                // rows of a pass
    uint4* pool = static_cast<uint4*>(is_v ? P.pool[1] : P.pool[0]) + (size_t)g * P.row_vecs +
                  (kind - (is_v ? P.slices : 0)) * lanes + tid % lanes;
    const int64_t stride = (int64_t)P.h_kv * P.row_vecs;
    compact_walk<U, uint4, int>(
        keep, new_len, L, per, tid / lanes < per ? tid / lanes : -1, tid % lanes == 0,
        P.error_word,
        [&](int j) {
          const CompactPlace p = compact_place(P, table, j);
          return p.page < 0 ? -1 : p.page * P.page_size + p.off;
        },
        [&](int slot) { return pool + slot * stride; });
  } else if (P.scale[0] && kind < 2 * P.slices + 2) {
    float* scale = (kind == 2 * P.slices ? P.scale[0] : P.scale[1]) + (size_t)g * P.page_size;
    compact_walk<U, float, int64_t>(
        keep, new_len, L, T, tid, false, nullptr,
        [&](int j) -> int64_t {
          const CompactPlace p = compact_place(P, table, j);
          return p.page < 0 ? -1 : (int64_t)p.page * P.h_kv * P.page_size + p.off;
        },
        [&](int64_t slot) { return scale + slot; });
  } else {
    float* m = P.mass + (size_t)row * P.mass_len;
    compact_walk<U, float, int>(
        keep, new_len, L, T, tid, false, nullptr, [&](int j) { return j; },
        [&](int j) { return m + j; });
    // positions that no key holds any more gather nothing; the last batch's
    // loads are behind the walk's barrier
    __syncthreads();
    for (int j = new_len + tid; j < L; j += T) m[j] = 0.f;
  }
}

// ------------------------------------------- compact, positions closed up --
//
// The same move with every K row turned by the positions it moves.  All that
// moves of a (sequence, KV head) is moved by one cluster of CTAs in one walk:
// batches of positions are shared out among its CTAs and their rows' rotary
// units (rope.cuh) among a row's threads, each of which takes the same words
// of the K row and of the V row; the row's first thread takes the scales and
// the mass.  So the list, the table and the checks are read once for all of it,
// and every CTA has arithmetic (a row that moves has an angle of its own for
// every pair) beside its loads.  A batch's rows are loaded while the batch
// before it is turned (its list entries come three batches ahead, its pages
// two); its stores come behind a barrier of the cluster that every thread
// reaches with its rows loaded: positions below the batch's end, which no later
// batch reads (every keep[j] >= j), as above.
// Bound: HBM where rows are many, 2 x (K and V row) per moved row: 64 bf16
// sequences of 512-8,192 keys cut to 2,048 take 151 us (858 MB, 5.7 TB/s; the
// move alone 151), against 250 with K and V moved by CTAs of their own (the
// index work twice, CTAs of K four times as long as those of V) and 169 where
// pages were looked up in the batch that reads them.  f32 rows 304 us (1.7 GB,
// 5.6 TB/s).  One-byte rows are bound by instructions, 420 a warp and unit: e4m3
// 134 us (431 MB), int8 233 (a scale, 16 quotients and their checks more; two
// units a thread spilled or left two CTAs an SM: 135-157 and 240-253 us).
// One sequence of 32,768 cut to 8,192 takes 25 us, 24 of up to 8,192 e4m3 keys
// cut to 1,500 30 us: a batch's latency (some 2.5 us of loads, turns and the
// cluster's barrier) times their number.  (The barrier is arrived at before the
// next batch's loads, which its release would wait for: 2-9% less.)
struct CompactTurn {
  const uint64_t* freqs;
  int32_t rot, interleaved;
  int32_t units, slices;  // rotary units of a row, clusters that share a row
  int32_t cluster;        // CTAs of a cluster
};

// A row's units here: rot is a multiple of 16 too, so in the layout of halves a
// unit turns as a whole (u < rot / 16: its lower words rot/4 apart, for W = 4) or
// lies as a whole behind the rotated part; interleaved as in rope_unit_words.
template <bool INTER, int W>
struct CompactUnits {
  static constexpr int NW = 16 / W, n = INTER ? W / 2 : W;
  static TL_DEVINLINE void words(int u, int d, int rot, int* at) {
    if (!INTER && 16 * u < rot) {
#pragma unroll
      for (int w = 0; w < NW; ++w)
        at[w] = W * u + (w % (NW / 2)) * (rot >> 2) + (w >= NW / 2 ? rot >> 1 : 0);
    } else {
      const int from = INTER ? 0 : rot;
#pragma unroll
      for (int w = 0; w < NW; ++w) at[w] = from + w * ((d - from) / NW) + W * (u - (from >> 4));
    }
  }
  // whether pair k turns, and its index
  static TL_DEVINLINE bool turn(const int* at, int k, int u, int rot) {
    return INTER ? at[k / n] < rot : 16 * u < rot;
  }
  static TL_DEVINLINE int index(const int* at, int k) {
    return (INTER ? at[k / n] >> 1 : at[k / n]) + k % n;
  }
  // the unit's values turned back by m positions, two pairs at once
  static TL_DEVINLINE void turn_back(float* x, const int* at, int u, int rot,
                                     const uint64_t* freqs, uint32_t m) {
    uint64_t f[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) f[k] = turn(at, k, u, rot) ? __ldg(freqs + index(at, k)) : 0;
#pragma unroll
    for (int k = 0; k < 8; k += 2) {
      if (!turn(at, k, u, rot)) continue;
      float2 a, b;
      rope_turns(f[k], f[k + 1], m, a, b);
      float &la = INTER ? x[2 * k] : x[k], &ha = INTER ? x[2 * k + 1] : x[8 + k];
      float &lb = INTER ? x[2 * k + 2] : x[k + 1], &hb = INTER ? x[2 * k + 3] : x[9 + k];
      const uint64_t lo = f2_pack(la, lb), hi = f2_pack(ha, hb), c = f2_pack(a.x, b.x);
      const float2 l = f2_unpack(f2_fma(lo, c, f2_mul(hi, f2_pack(a.y, b.y))));
      const float2 h = f2_unpack(f2_fma(hi, c, f2_mul(lo, f2_pack(-a.y, -b.y))));
      la = l.x, lb = l.y, ha = h.x, hb = h.y;
    }
  }
};

template <int E>
struct CompactRow {
  static constexpr int W = E == kElemF32 ? 4 : 8;
  RopeUnit<E, W> k, v;
  float k_scale, v_scale, mass;
};

constexpr int kCompactRopeThreads = 256;
template <int E, bool INTER>
__global__ void __launch_bounds__(kCompactRopeThreads, E == kElemF32 ? 2 : 3)
    compact_rope_kernel(CompactParams P, CompactTurn R) {
  constexpr int W = CompactRow<E>::W, T = kCompactRopeThreads;
  using Units = CompactUnits<INTER, W>;
  const int tid = threadIdx.x;
  const int group = (int)blockIdx.x / R.cluster, rank = (int)blockIdx.x - group * R.cluster;
  const int row = group / R.slices, slice = group - row * R.slices;
  const int b = row / P.h_kv, g = row - b * P.h_kv;
  const int L = P.context_lens[b], new_len = P.new_lens[b];
  const int64_t cap = (int64_t)P.max_pages_per_seq * P.page_size;
  if (L > cap || (P.mass && L > P.mass_len) || new_len < 0 || new_len > P.n ||
      new_len > max(L, 0)) {  // the sequence stays as it is (all of the cluster leaves)
    if (rank == 0 && tid == 0) report(P.error_word, TL_DEVERR_CONTEXT_RANGE);
    return;
  }
  const int32_t* keep = P.keep + (size_t)row * P.n;
  const int32_t* table = P.block_table + (size_t)b * P.max_pages_per_seq;
  const int lanes = R.units / R.slices, per = T / lanes;  // threads of a row, rows of a pass
  const int u = slice * lanes + tid % lanes;
  const int batch = per * R.cluster, r = rank * per + tid / lanes;
  const bool mine = tid / lanes < per, first = u == 0;
  int at[16 / W];
  Units::words(u, R.units * 16, R.rot, at);
  const int64_t row_bytes = (int64_t)P.row_vecs * 16, stride = P.h_kv * row_bytes;
  char* k = static_cast<char*>(P.pool[0]) + g * row_bytes;
  char* v = static_cast<char*>(P.pool[1]) + g * row_bytes;
  float* mass = P.mass ? P.mass + (size_t)row * P.mass_len : nullptr;
  auto scale_at = [&](int slot) {  // int8: [num_pages][h_kv][page_size]
    const int page = P.ps_shift >= 0 ? slot >> P.ps_shift : slot / P.page_size;
    return ((int64_t)page * (P.h_kv - 1) + g) * P.page_size + slot;
  };
  // the list's entry for position j
  auto entry = [&](int j) { return mine && j < new_len ? __ldg(keep + j) : j; };
  auto block_of = [&](int j) { return P.ps_shift >= 0 ? j >> P.ps_shift : j / P.page_size; };
  // the pages that hold positions s and j; read here, looked at a batch later
  auto pages = [&](int j, int s, int& from, int& to) {
    from = to = -1;
    if (s <= j || s >= L) return;
    from = __ldg(table + block_of(s));
    to = __ldg(table + block_of(j));
  };
  // the slots that entry s moves position j's row from and to, in place of the
  // pages; to < 0: none
  auto places = [&](int j, int s, int& from, int& to) {
    if (s == j) return;  // stays, or not a row of this thread
    if (s < j || s >= L) {
      if (first) report(P.error_word, TL_DEVERR_CONTEXT_RANGE);
      return;
    }
    if (from < 0 || from >= P.num_pages || to < 0 || to >= P.num_pages) {
      if (first) report(P.error_word, TL_DEVERR_PAGE_RANGE);
      to = -1;
      return;
    }
    from = from * P.page_size + (s - block_of(s) * P.page_size);
    to = to * P.page_size + (j - block_of(j) * P.page_size);
  };
  auto load = [&](CompactRow<E>& x, int s, int from, int to) {
    if (to < 0) return;
    x.k.load(k + from * stride, at);
    x.v.load(v + from * stride, at);
    if (E == kElemInt8) {
      x.k_scale = __ldcg(P.scale[0] + scale_at(from));
      if (first) x.v_scale = __ldcg(P.scale[1] + scale_at(from));
    }
    if (mass && first) x.mass = __ldcg(mass + s);
  };
  CompactRow<E> x, y;
  int s = entry(r), s1 = entry(batch + r), s2 = entry(2 * batch + r);
  int from, to, from1, to1;
  pages(r, s, from, to);
  pages(batch + r, s1, from1, to1);
  places(r, s, from, to);
  load(x, s, from, to);
  for (int j = r; j - r < new_len; j += batch) {
    // this thread's row of the batch is loaded (the release is behind the load);
    // what it loads from here on is for later batches
    if (R.cluster > 1) asm volatile("barrier.cluster.arrive.release.aligned;\n" ::: "memory");
    // the next batch's row, the pages of the one behind it, the entry of a third
    places(j + batch, s1, from1, to1);
    load(y, s1, from1, to1);
    int from2, to2;
    pages(j + 2 * batch, s2, from2, to2);
    const int s3 = entry(j + 3 * batch);
    bool bad = false;
    if (E == kElemInt8 || (to >= 0 && Units::turn(at, 0, u, R.rot))) {
      float z[16];
      x.k.values(z);
      if constexpr (E == kElemInt8) {
#pragma unroll
        for (int e = 0; e < 16; ++e) z[e] *= x.k_scale;
      }
      if (to >= 0) Units::turn_back(z, at, u, R.rot, R.freqs, (uint32_t)(s - j));
      if constexpr (E == kElemInt8) {
        float m = to >= 0 ? rope_unit_max(z, bad) : 0.f;
        for (int o = lanes >> 1; o > 0; o >>= 1)
          m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        x.k_scale = __fdiv_rn(m, 127.f);
        x.k.set_codes(z, x.k_scale, !bad);
      } else {
        const RopeUnit<E, W> was = x.k;
        x.k.set(z);
        if (INTER) {  // words behind the rotated part keep their bits
#pragma unroll
          for (int w = 0; w < 16 / W; ++w)
            if (at[w] >= R.rot) x.k.w[w] = was.w[w];
        }
      }
    }
    if (E == kElemInt8 && bad) report(P.error_word, TL_DEVERR_VALUE_RANGE);
    // every thread's row of this batch is loaded before any of it is stored
    if (R.cluster > 1) asm volatile("barrier.cluster.wait.acquire.aligned;\n" ::: "memory");
    else __syncthreads();
    if (to >= 0) {
      x.k.store(k + to * stride, at);
      x.v.store(v + to * stride, at);
      if (E == kElemInt8 && first) {
        P.scale[0][scale_at(to)] = x.k_scale;
        P.scale[1][scale_at(to)] = x.v_scale;
      }
      if (mass && first) mass[j] = x.mass;
    }
    x = y;
    s = s1, s1 = s2, s2 = s3;
    to = to1, from1 = from2, to1 = to2;
  }
  // positions that no key holds any more gather nothing (the masses that move
  // are loaded: the last batch's barrier is past)
  if (mass && slice == 0)
    for (int j = new_len + rank * T + tid; j < L; j += R.cluster * T) mass[j] = 0.f;
}

// Whether the current device holds a cluster of 16 of the int8 kernel's CTAs
// (more than every device has to; asked once a device).
template <bool INTER>
static bool holds_16(cudaLaunchConfig_t cfg) {
  static std::atomic<int> known[64];  // 0: not asked
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return false;
  if (known[dev].load() == 0) {
    auto kern = compact_rope_kernel<kElemInt8, INTER>;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 16;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.gridDim = dim3(16);
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int n = 0;
    const bool ok =
        cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) ==
            cudaSuccess &&
        cudaOccupancyMaxActiveClusters(&n, kern, &cfg) == cudaSuccess && n > 0;
    if (!ok) cudaGetLastError();
    known[dev].store(ok ? 1 : -1);
  }
  return known[dev].load() > 0;
}

static cudaError_t launch_compact_rope(const CompactParams& P, CompactTurn R, int64_t rows, int d,
                                       int elem, cudaStream_t st) {
  R.units = d / 16;
  const bool i8 = P.scale[0] != nullptr;
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(kCompactRopeThreads);
  cfg.stream = st;
  // Few rows are shared by clusters of up to 8 CTAs, and by slices of a row
  // (whole 32-byte sectors of words; an int8 row is one slice, for its scale),
  // while every CTA has a place at once: three on an SM, f32 ones two.  8 rows of
  // 8,192 kept keys take 70 us with clusters of 8, 40 with two slices, 25 with
  // four (int8, one slice: 75, and 46 with the clusters of 16 that this GPU
  // holds); 128 rows of 2,048 78 us with clusters of 2, 61 with 3; 96 rows of
  // 1,500 e4m3 keys 49 with 2, 30 with 4, 33 with 8 (two waves).
  const int64_t ctas = (int64_t)num_sms() * (elem == 4 ? 2 : 3);
  const bool wide = i8 && rows * 16 <= num_sms() &&
                    (R.interleaved ? holds_16<true>(cfg) : holds_16<false>(cfg));
  R.cluster = (int)std::min<int64_t>(wide ? 16 : 8, std::max<int64_t>(1, ctas / rows));
  R.slices = 1;
  const int least = elem == 1 ? 4 : 2;
  while (!i8 && R.units % (2 * R.slices) == 0 && R.units / (2 * R.slices) >= least &&
         rows * R.cluster * 2 * R.slices <= ctas)
    R.slices *= 2;
  auto kern = R.interleaved ? (i8          ? compact_rope_kernel<kElemInt8, true>
                               : elem == 1 ? compact_rope_kernel<kElemE4m3, true>
                               : elem == 2 ? compact_rope_kernel<kElemBf16, true>
                                           : compact_rope_kernel<kElemF32, true>)
                            : (i8          ? compact_rope_kernel<kElemInt8, false>
                               : elem == 1 ? compact_rope_kernel<kElemE4m3, false>
                               : elem == 2 ? compact_rope_kernel<kElemBf16, false>
                                           : compact_rope_kernel<kElemF32, false>);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = R.cluster;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.gridDim = dim3((unsigned)(rows * R.slices * R.cluster));
  cfg.attrs = attr;
  cfg.numAttrs = R.cluster > 1 ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kern, P, R);
}

static tl_status compact_impl(void* k, void* v, float* k_scales, float* v_scales,
                              const int32_t* block_table, int32_t max_pages_per_seq,
                              const int32_t* context_lens, const int32_t* keep, int32_t n_keep,
                              const int32_t* new_lens, float* mass, int32_t mass_len, int32_t B,
                              int32_t h_kv, int32_t d, int32_t num_pages, int32_t page_size,
                              int elem, uint32_t* error_word, void* stream,
                              const CompactTurn* turn = nullptr) {
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
  if (turn) {
    // the lists are read while other CTAs write
    const size_t lens = sizeof(int32_t) * (size_t)B;
    const struct {
      const void* p;
      size_t bytes;
    } read[] = {{block_table, lens * max_pages_per_seq},
                {context_lens, lens},
                {keep, lens * h_kv * n_keep},
                {new_lens, lens},
                {turn->freqs, sizeof(uint64_t) * (size_t)(turn->rot / 2)}};
    for (const auto& m : moved)
      for (const auto& r : read)
        if (m.bytes && overlap(m.p, m.bytes, r.p, r.bytes)) return TL_ERR_INVALID_ARG;
  }
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
  if (turn)
    return launch_compact_rope(P, *turn, rows, d, elem, (cudaStream_t)stream) == cudaSuccess
               ? launch_status()
               : TL_ERR_CUDA;
  P.slices = 1;
  while (P.row_vecs % (2 * P.slices) == 0 && P.row_vecs / (2 * P.slices) >= 2 &&
         rows * 2 * P.slices < 2 * num_sms())
    P.slices *= 2;
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
  const tl::CompactTurn turn = {freqs, rot_dim, interleaved != 0, 0, 0, 0};
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
  const tl::CompactTurn turn = {freqs, rot_dim, interleaved != 0, 0, 0, 0};
  return tl::compact_impl(k_codes, v_codes, k_scales, v_scales, block_table, max_pages_per_seq,
                          context_lens, keep, n_keep, new_lens, mass, mass_len, B, h_kv, d,
                          num_pages, page_size, 1, error_word, stream, &turn);
}
