// The n largest of each row of f32 values, in ascending index order: the
// selection shared by the page selection (a row of page scores) and the
// eviction (a row of accumulated weights).
//
// A row has `len` values and `n` places.  With len <= n every index is taken.
// Otherwise the first `first` and the last `last` indices are taken whatever
// their values, and the other n - first - last places go to the largest
// values of the middle, equal values to the lowest index; a NaN ranks below
// everything.  The values are compared as unsigned keys in the floats' order
// (+0 and -0 are one key), so the result is exact and does not depend on how
// the row is split.
//
// Method: what is sought is one (key, index) pair, the last one taken; then an
// index is taken when its key is larger, or equal with an index not behind.
// A radix selection narrows the range of keys that holds it: the smallest and
// largest key are found first, the range between them is cut into 1,024 to 4,096
// equal bins (linear in the key, so about even over a heavy-tailed row's
// values), a histogram in shared memory tells the bin, and that bin is cut
// again until it holds at most 128 values, which are ranked against each
// other (once, for rows of some 10,000 spread values).  Where the bin is one
// key (a row of equal values) the search goes on over the indices.
//
// Layout: a row is one cluster of 1-8 CTAs, their histograms summed through
// distributed shared memory.  A CTA keeps its slice's keys in shared memory
// (a value is read from memory once), a lane four of them at a time, so that
// a thread needs few registers: the steps of one row are short sweeps between
// barriers, bound by instructions and by the barriers' latency, not by the
// values' bytes.  Slices past the shared memory read their values again.
//
// Measured on GB300: 512 rows of 1,024-32,768 masses (35 MB) 39 us, 8 rows of
// 131,072 (clusters of 4) 21 us.  Of the 39, loading and the extremes take 13,
// the histogram 8, the sweep for the bin's values 7, ranking them 3, placing 8;
// the schedulers issue 60% of the time: a warp has 4 steps of 128 values a
// sweep, and as many instructions around them.  Tried and no faster: halves of
// the keys in 16 bits (three rows an SM; 8-20% more for short rows), 512
// threads a row (46 us), 16,384 keys a CTA and clusters of 2 (a cluster's
// barriers and remote reads cost 2-5 thousand cycles each), the longest rows
// first (39.1 for 43 us then, before its own cost), ballots into a bit mask
// for the places, unrolling the sweeps less, twice the loads in flight (1%).
#pragma once

#include <cooperative_groups.h>

#include "common.cuh"

namespace tl {

// Bins of a pass: four a thread (1,024 to 4,096), so that a short row, which
// needs few, clears and scans few.
__host__ __device__ constexpr int select_bin_bits(int threads) {
  return threads >= 1024 ? 12 : threads >= 512 ? 11 : 10;
}
constexpr int kSelRank = 128;        // values ranked against each other at the end
constexpr int kSelKeysMax = 32768;   // keys of a slice kept in shared memory (128 KiB)
constexpr int kSelClusterMax = 8;

// Keys: 0 no value (behind the row), 1 NaN, then the floats in order (-0 =
// +0), all ones an index that is taken whatever its value.
constexpr uint32_t kSelForced = 0xffffffffu;
TL_DEVINLINE uint32_t select_key_number(float x) {  // x is not NaN
  const uint32_t u = __float_as_uint(x + 0.f);      // -0 + 0 is +0
  return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}
TL_DEVINLINE uint32_t select_key(float x) { return x != x ? 1u : select_key_number(x); }

template <int T>
struct SelectShared {
  static constexpr int kBinBits = select_bin_bits(T), kBins = 1 << kBinBits;
  static_assert(kBins == 4 * T, "a thread takes four bins");
  __align__(16) uint32_t hist[kBins + 32];  // the last 32: values outside a pass's range
  uint32_t minmax[2];     // this CTA's smallest and largest key
  uint32_t total;         // this CTA's taken values
  uint32_t tmp[2][32];    // block scans, alternating
  uint32_t found[3];      // bin, values above it, values in it
  uint32_t n_cand;        // (rank 0's are used) the values ranked at the end
  uint32_t cand[2][kSelRank];  // their keys and indices
  uint32_t last[2];       // key and index of the last value taken
};

// The block's exclusive scan of x in thread order; every thread gets the
// total.  One barrier; `tmp` must not be the previous scan's.
TL_DEVINLINE uint32_t select_block_scan(uint32_t x, uint32_t* tmp, uint32_t& total) {
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5, nw = blockDim.x >> 5;
  uint32_t inc = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t y = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += y;
  }
  if (lane == 31) tmp[wid] = inc;
  __syncthreads();
  const uint32_t mine = lane < nw ? tmp[lane] : 0u;
  uint32_t all = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t y = __shfl_up_sync(0xffffffffu, all, o);
    if (lane >= o) all += y;
  }
  total = __shfl_sync(0xffffffffu, all, 31);
  return __shfl_sync(0xffffffffu, all - mine, wid) + inc - x;
}

// One row x[0 .. len), by the CTAs of one cluster (rank `rank` of `csize`, a
// power of two; csize 1 needs no cluster launch), T threads each.  keys: key_cap words of
// 16-byte aligned shared memory, a multiple of 128 (FITS: no slice is longer).  emit(pos, i): index i is
// taken at place pos; tail(pos): place pos stays empty.  Returns the places
// that this CTA filled, first and one past the last ({0, 0} where len <= n:
// each thread filled places rank * T + tid, + csize * T, ...).
template <int T, bool FITS, class Emit, class Tail>
__device__ int2 select_row(SelectShared<T>& sh, uint32_t* keys, int key_cap, const float* x, int len,
                           int n, int first, int last, int rank, int csize, Emit emit,
                           Tail tail) {
  namespace cg = cooperative_groups;
  constexpr int NW = T / 32, PER = 4;
  constexpr int kSelBins = SelectShared<T>::kBins, kSelBinBits = SelectShared<T>::kBinBits;
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
  auto cluster_sync = [&]() {
    if (csize > 1) cg::this_cluster().sync();
    else __syncthreads();
  };
  auto peer = [&](uint32_t* p, int r) -> uint32_t* {
    return csize > 1 ? cg::this_cluster().map_shared_rank(p, r) : p;
  };
  if (len <= n) {  // everything
    for (int i = rank * T + tid; i < n; i += csize * T) {
      if (i < len) emit(i, i);
      else tail(i);
    }
    return make_int2(0, 0);  // every CTA of the cluster: no barrier is left waiting
  }
  // this CTA's slice of the row, and this warp's run of it: whole steps of 128
  // values, four neighbours a lane
  const int slice = (((len + csize - 1) >> (31 - __clz(csize))) + 127) / 128 * 128;
  const int i0 = min(rank * slice, len), i1 = min(i0 + slice, len);
  const int run = ((i1 - i0 + NW - 1) / NW + 127) / 128 * 128;
  const int w0 = i0 + min(wid * run, i1 - i0), w1 = min(w0 + run, i1);
  const int m0 = first, m1 = len - last;  // the middle: ranked by value
  const bool vec = (reinterpret_cast<uintptr_t>(x + i0) & 15u) == 0;
  auto load4 = [&](int i) {
    if (vec && i + 3 < len) return __ldcg(reinterpret_cast<const float4*>(x + i));
    float4 f;
    f.x = i < len ? __ldcg(x + i) : 0.f;
    f.y = i + 1 < len ? __ldcg(x + i + 1) : 0.f;
    f.z = i + 2 < len ? __ldcg(x + i + 2) : 0.f;
    f.w = i + 3 < len ? __ldcg(x + i + 3) : 0.f;
    return f;
  };
  auto key_of = [&](float f, int i) {
    return i >= len ? 0u : i < m0 || i >= m1 ? kSelForced : select_key(f);
  };
  auto keys_of = [&](const float4& f, int i) {
    return make_uint4(key_of(f.x, i), key_of(f.y, i + 1), key_of(f.z, i + 2), key_of(f.w, i + 3));
  };
  // a lane reads back the keys it stored; behind a barrier, any of its warp's
  auto keys_at = [&](int i) {
    return FITS || i - i0 < key_cap ? *reinterpret_cast<const uint4*>(keys + (i - i0))
                            : keys_of(load4(i), i);
  };
  auto key_at = [&](int i) {
    return FITS || i - i0 < key_cap ? keys[i - i0] : i < len ? key_of(__ldcg(x + i), i) : 0u;
  };

  auto clear_hist = [&]() {
    for (int b = tid; b < kSelBins / 4; b += T)
      reinterpret_cast<uint4*>(sh.hist)[b] = make_uint4(0u, 0u, 0u, 0u);
  };
  clear_hist();
  if (tid == 0) {
    sh.n_cand = 0u;
    sh.minmax[0] = kSelForced;
    sh.minmax[1] = 0u;
  }
  uint32_t kmin = kSelForced, kmax = 0u;
  constexpr int U = 4;  // loads in flight
  for (int w = w0; w < w1; w += 128 * U) {
    float4 f[U];
#pragma unroll
    for (int u = 0; u < U; ++u) f[u] = load4(w + 128 * u + 4 * lane);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int ws = w + 128 * u, i = ws + 4 * lane;
      if (ws >= w1) break;
      uint4 k;
      if (ws >= m0 && ws + 128 <= m1) {  // all of the step is in the middle
        k = make_uint4(select_key_number(f[u].x), select_key_number(f[u].y),
                       select_key_number(f[u].z), select_key_number(f[u].w));
        const float any = (f[u].x + f[u].y) + (f[u].z + f[u].w);
        if (any != any)  // a NaN (or opposite infinities) among the four
          k = make_uint4(select_key(f[u].x), select_key(f[u].y), select_key(f[u].z),
                         select_key(f[u].w));
        kmin = min(min(min(kmin, k.x), min(k.y, k.z)), k.w);
        kmax = max(max(max(kmax, k.x), max(k.y, k.z)), k.w);
      } else {
        k = keys_of(f[u], i);
        const uint32_t kk[4] = {k.x, k.y, k.z, k.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (kk[j] - 1u < kSelForced - 1u) {  // neither none nor forced
            kmin = min(kmin, kk[j]);
            kmax = max(kmax, kk[j]);
          }
        }
      }
      if (FITS || i - i0 < key_cap) *reinterpret_cast<uint4*>(keys + (i - i0)) = k;
    }
  }
  kmin = __reduce_min_sync(0xffffffffu, kmin);
  kmax = __reduce_max_sync(0xffffffffu, kmax);
  __syncthreads();
  if (lane == 0) {
    atomicMin(&sh.minmax[0], kmin);
    atomicMax(&sh.minmax[1], kmax);
  }
  cluster_sync();
  kmin = sh.minmax[0];
  kmax = sh.minmax[1];
  if (csize > 1) {
#pragma unroll
    for (int r = 0; r < kSelClusterMax; ++r) {
      if (r < csize) {
        const uint32_t* m = peer(sh.minmax, r);
        kmin = min(kmin, m[0]);
        kmax = max(kmax, m[1]);
      }
    }
  }

  // The search: the need-th largest of the cnt values in lo .. lo + span.
  // by_index: among the values of key `equal`, over len - 1 - index.
  uint32_t need = (uint32_t)(n - first - last), cnt = (uint32_t)(m1 - m0);
  uint32_t lo = kmin, span = kmax - kmin, equal = 0u;
  bool by_index = false;
  uint32_t count = 0;  // this warp's taken values, once `counted`
  bool counted = false;
  // the last pair taken; none so far: above every value, below the forced
  uint32_t last_key = kSelForced - 1u;
  int last_idx = -1;
  // f(index, key) for this warp's values that the range may hold
  auto each = [&](auto f) {
#pragma unroll 4
    for (int w = w0; w < w1; w += 128) {
      const int i = w + 4 * lane;
      const uint4 k = keys_at(i);
      f(i, k.x);
      f(i + 1, k.y);
      f(i + 2, k.z);
      f(i + 3, k.w);
    }
  };
  // places of equal keys: from the row's end, so that the lowest is the largest
  auto place = [&](int i) { return (uint32_t)(len - 1 - i); };
  for (int pass = 0; need > 0; ++pass) {
    if (need == cnt) {  // all of the range
      last_key = by_index ? equal : lo;
      last_idx = by_index ? len - 1 - (int)lo : len;
      break;
    }
    if (cnt <= (uint32_t)kSelRank) {  // rank them
      uint32_t* n_cand = peer(&sh.n_cand, 0);
      uint32_t* cand = peer(&sh.cand[0][0], 0);
      if (by_index) {
        each([&](int i, uint32_t k) {
          if (k != equal || place(i) - lo > span) return;
          const uint32_t at = atomicAdd(n_cand, 1u);
          if (at < (uint32_t)kSelRank) {
            cand[at] = k;
            cand[kSelRank + at] = (uint32_t)i;
          }
        });
      } else {  // the same sweep counts the values above the range
        counted = true;
        const uint32_t hi = lo + span;
        // a lane keeps the last two it meets and lists them behind the sweep
        // (listing each as it is met stalls the warp every other step); one
        // that meets more walks its values again
        uint32_t met = 0u;
        int x0 = 0, x1 = 0;
        each([&](int i, uint32_t k) {
          count += k > hi ? 1u : 0u;
          const bool in = k - lo <= span;
          x1 = in ? x0 : x1;
          x0 = in ? i : x0;
          met += in ? 1u : 0u;
        });
        auto list = [&](uint32_t k, int i) {
          const uint32_t at = atomicAdd(n_cand, 1u);
          if (at < (uint32_t)kSelRank) {
            cand[at] = k;
            cand[kSelRank + at] = (uint32_t)i;
          }
        };
        if (met == 1u || met == 2u) list(key_at(x0), x0);
        if (met == 2u) list(key_at(x1), x1);
        if (met > 2u)
          for (int i = w0 + 4 * lane; i < w1; i += 128) {
            const uint4 k = keys_at(i);
            const uint32_t kk[4] = {k.x, k.y, k.z, k.w};
            for (int j = 0; j < 4; ++j)
              if (kk[j] - lo <= span) list(kk[j], i + j);
          }
      }
      cluster_sync();
      uint32_t* ck = &sh.cand[0][0];
      if (csize > 1 && rank != 0) {  // a copy of rank 0's list
        for (int c = tid; c < (int)cnt; c += T) {
          ck[c] = cand[c];
          ck[kSelRank + c] = cand[kSelRank + c];
        }
        __syncthreads();
      }
      // T / kSelRank threads a value, each against its share of the others
      constexpr int kShare = T / kSelRank;
      const int mine = tid / kShare;
      uint32_t k = 0u, at = 0u, better = 0u;
      if (mine < (int)cnt) {
        k = ck[mine];
        at = ck[kSelRank + mine];
#pragma unroll 4
        for (int c = tid % kShare; c < (int)cnt; c += kShare)
          better += ck[c] > k || (ck[c] == k && ck[kSelRank + c] < at) ? 1u : 0u;
      }
#pragma unroll
      for (int o = 1; o < kShare; o <<= 1) better += __shfl_xor_sync(0xffffffffu, better, o);
      if (mine < (int)cnt && better == need - 1) {  // its threads write the same
        sh.last[0] = k;
        sh.last[1] = at;
      }
      __syncthreads();
      last_key = sh.last[0];
      last_idx = (int)sh.last[1];
      if (counted)  // the ranked values that are taken and this warp's
        for (int c = lane; c < (int)cnt; c += 32) {
          const int i = (int)ck[kSelRank + c];
          if (i >= w0 && i < w1 && (ck[c] > last_key || (ck[c] == last_key && i <= last_idx)))
            ++count;
        }
      break;
    }
    if (span == 0u && !by_index) {  // one key: on over the indices
      by_index = true;
      equal = lo;
      lo = 0u;
      span = (uint32_t)(len - 1);
    }
    const int bits = 32 - __clz(span);
    const int shift = bits > kSelBinBits ? bits - kSelBinBits : 0;
    if (pass > 0) {
      if (csize > 1) cg::this_cluster().sync();  // peers are past the last pass's histogram
      clear_hist();
      __syncthreads();
    }
    uint32_t* hist = sh.hist;
    if (!by_index) {
      // a value outside the range counts in a spare bin of its lane: fewer
      // instructions than a branch around the count
      const uint32_t spare = (uint32_t)(kSelBins + lane);
      each([&](int, uint32_t k) {
        atomicAdd(hist + (k - lo <= span ? (k - lo) >> shift : spare), 1u);
      });
    } else {
      each([&](int i, uint32_t k) {
        if (k == equal && place(i) - lo <= span) atomicAdd(hist + ((place(i) - lo) >> shift), 1u);
      });
    }
    cluster_sync();
    // from the top bin down: thread t takes the PER bins that end below
    // kSelBins - t * PER
    const int b0 = kSelBins - (tid + 1) * PER;
    uint32_t c[PER], sum = 0;
#pragma unroll
    for (int j = 0; j < PER; ++j) c[j] = 0u;
    if (csize > 1) {
#pragma unroll
      for (int r = 0; r < kSelClusterMax; ++r) {
        if (r < csize) {
          const uint4* h = reinterpret_cast<const uint4*>(peer(hist, r) + b0);
#pragma unroll
          for (int j = 0; j < PER / 4; ++j) {
            const uint4 v = h[j];
            c[4 * j] += v.x;
            c[4 * j + 1] += v.y;
            c[4 * j + 2] += v.z;
            c[4 * j + 3] += v.w;
          }
        }
      }
    } else {
#pragma unroll
      for (int j = 0; j < PER; ++j) c[j] = hist[b0 + j];
    }
#pragma unroll
    for (int j = 0; j < PER; ++j) sum += c[j];
    uint32_t total;
    uint32_t before = select_block_scan(sum, sh.tmp[pass & 1], total);
    if (before < need && need <= before + sum) {
      uint32_t bin = 0, above = 0, in = 0;
#pragma unroll
      for (int j = PER - 1; j >= 0; --j) {
        if (before < need && need <= before + c[j]) {
          bin = (uint32_t)(b0 + j);
          above = before;
          in = c[j];
        }
        before += c[j];
      }
      sh.found[0] = bin;
      sh.found[1] = above;
      sh.found[2] = in;
    }
    __syncthreads();
    const uint32_t bin = sh.found[0];
    need -= sh.found[1];
    cnt = sh.found[2];
    lo += bin << shift;
    span = min(span - (bin << shift), (1u << shift) - 1u);
  }

  auto taken = [&](uint32_t k, int i) {
    return k > last_key || (k == last_key && i <= last_idx);
  };
  // Place the taken values in index order: each warp's count (most came with
  // the last sweep), a scan over the warps, the cluster's earlier CTAs.
  if (!counted) {
    each([&](int i, uint32_t k) { count += taken(k, i) ? 1u : 0u; });
  }
  count = __reduce_add_sync(0xffffffffu, count);
  __syncthreads();  // sh.tmp is free
  uint32_t total;
  int at = (int)select_block_scan(lane == 0 ? count : 0u, sh.tmp[0], total);
  at = __shfl_sync(0xffffffffu, at, 0);
  int base = 0;
  if (csize > 1) {
    if (tid == 0) sh.total = total;
    cg::this_cluster().sync();
#pragma unroll
    for (int r = 0; r < kSelClusterMax; ++r)
      if (r < rank) base += (int)*peer(&sh.total, r);
    at += base;
    // no peer's shared memory is read behind this point
    asm volatile("barrier.cluster.arrive.release.aligned;\n" ::: "memory");
  }
  const uint32_t below = (1u << lane) - 1u;
  const int end = at + (int)count;
  for (int w = w0; w < w1 && at < end; w += 128) {
    // a lane's values 32 apart: a ballot orders them, and the warp's stores
    // run together
    const int i = w + lane;
    uint32_t k[4], m[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) k[j] = key_at(i + 32 * j);
    if (w <= last_idx && last_idx < w + 128) {  // the step of the last one taken
#pragma unroll
      for (int j = 0; j < 4; ++j) m[j] = __ballot_sync(0xffffffffu, taken(k[j], i + 32 * j));
    } else {  // equal values are all taken before it, and none behind it
      const uint32_t over = w > last_idx ? last_key : last_key - 1u;  // last_key >= 1
#pragma unroll
      for (int j = 0; j < 4; ++j) m[j] = __ballot_sync(0xffffffffu, k[j] > over);
    }
    if ((m[0] | m[1] | m[2] | m[3]) == 0u) continue;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (m[j] >> lane & 1u) emit(at + __popc(m[j] & below), i + 32 * j);
      at += __popc(m[j]);
    }
  }
  if (csize > 1)  // the CTA stays until its peers have read its totals
    asm volatile("barrier.cluster.wait.acquire.aligned;\n" ::: "memory");
  return make_int2(base, base + (int)total);
}

// Threads per CTA, CTAs per row and keys kept per CTA for `rows` rows of up to
// cap values.
struct SelectShape {
  int threads, cluster, keys;
  bool fits;  // every slice's keys are kept
};
SelectShape select_shape(int64_t rows, int64_t cap);
// Launch of a kernel over `rows` clusters (its forms: 256, 512 and 1,024
// threads, then 1,024 threads with slices that do not fit); dependent: a
// programmatic dependent of the stream's previous kernel.
cudaError_t launch_rows(const void* const (&kernels)[4], int64_t rows, const SelectShape& s,
                        void** args, bool dependent, cudaStream_t st);

}  // namespace tl
