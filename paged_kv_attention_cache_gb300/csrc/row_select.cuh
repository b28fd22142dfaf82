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
// Method: a radix selection over the keys' range.  One pass finds the row's
// smallest and largest key; the range between them is cut into 2,048 equal
// bins (linear in the key, so in the logarithm of the value), a histogram in
// shared memory finds the bin that the n-th value falls into, and that bin is
// cut again until its members are all taken or all equal.  Two or three
// passes do for any distribution, and a row whose values sit in registers is
// read from memory once.  A row is one cluster of 1-8 CTAs (its slices'
// histograms are summed through distributed shared memory); each CTA then
// counts its taken values, and ballots and one scan place them in index
// order.
#pragma once

#include <cooperative_groups.h>

#include "common.cuh"

namespace tl {

constexpr int kSelBins = 2048;
constexpr int kSelBinBits = 11;
constexpr int kSelRegs = 16;        // values a thread keeps in registers
constexpr int kSelMaxThreads = 1024;

// A value's key: unsigned order = float order, NaN lowest, -0 = +0.
TL_DEVINLINE uint32_t select_key(float x) {
  if (x != x) return 0u;
  const uint32_t u = __float_as_uint(x == 0.f ? 0.f : x);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

struct SelectShared {
  uint32_t hist[2][kSelBins];  // two, so that one is cleared while peers read the other
  uint32_t minmax[2];          // this CTA's smallest and largest key
  uint32_t totals[2];          // this CTA's taken values and values equal to the threshold
  uint32_t warp_a[32], warp_b[32];
  uint32_t found[3];           // bin, values above it, values in it
  uint32_t counts[kSelRegs][32];  // per round of one value a thread and warp: above | equal << 16
};

// The block's exclusive scan of x in thread order; every thread gets the total.
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
  uint32_t before = 0, all = 0;
  for (int w = 0; w < nw; ++w) {
    const uint32_t v = tmp[w];
    if (w < wid) before += v;
    all += v;
  }
  __syncthreads();  // tmp is reused
  total = all;
  return before + inc - x;
}

// One row, by the CTAs of one cluster (rank `rank` of `csize`; csize 1 needs
// no cluster launch).  value(i): the row's value i; emit(pos, i): index i is
// taken at place pos; tail(pos): place pos stays empty.
template <class Value, class Emit, class Tail>
__device__ void select_row(SelectShared& sh, int len, int n, int first, int last, int rank,
                           int csize, Value value, Emit emit, Tail tail) {
  namespace cg = cooperative_groups;
  const int tid = threadIdx.x, T = blockDim.x, lane = tid & 31, wid = tid >> 5, nw = T >> 5;
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
    return;  // the same for every CTA of the cluster: no barrier is left waiting
  }
  // this CTA's slice of the row, a multiple of 32 values long
  const int slice = ((len + csize - 1) / csize + 31) / 32 * 32;
  const int i0 = min(rank * slice, len), i1 = min(i0 + slice, len);
  const int m0 = first, m1 = len - last;  // the middle: ranked by value
  uint32_t reg[kSelRegs];
#pragma unroll
  for (int u = 0; u < kSelRegs; ++u) {
    const int i = i0 + u * T + tid;
    reg[u] = i < i1 ? select_key(value(i)) : 0u;
  }
  // f(i, key, in the slice) for this thread's values, steps of T apart, all
  // lanes of a warp together
  auto each = [&](auto f) {
#pragma unroll
    for (int u = 0; u < kSelRegs; ++u) {
      const int i = i0 + u * T + tid;
      f(i, reg[u], i < i1);
    }
    for (int w0 = i0 + kSelRegs * T + wid * 32; w0 < i1; w0 += T) {
      const int i = w0 + lane;
      f(i, i < i1 ? select_key(value(i)) : 0u, i < i1);
    }
  };

  for (int b = tid; b < 2 * kSelBins; b += T) (&sh.hist[0][0])[b] = 0u;
  uint32_t kmin = 0xffffffffu, kmax = 0u;
  each([&](int i, uint32_t k, bool in) {
    if (in && i >= m0 && i < m1) {
      kmin = min(kmin, k);
      kmax = max(kmax, k);
    }
  });
  kmin = __reduce_min_sync(0xffffffffu, kmin);
  kmax = __reduce_max_sync(0xffffffffu, kmax);
  if (lane == 0) {
    sh.warp_a[wid] = kmin;
    sh.warp_b[wid] = kmax;
  }
  __syncthreads();
  if (wid == 0) {
    kmin = __reduce_min_sync(0xffffffffu, lane < nw ? sh.warp_a[lane] : 0xffffffffu);
    kmax = __reduce_max_sync(0xffffffffu, lane < nw ? sh.warp_b[lane] : 0u);
    if (lane == 0) {
      sh.minmax[0] = kmin;
      sh.minmax[1] = kmax;
    }
  }
  cluster_sync();
  kmin = 0xffffffffu;
  kmax = 0u;
  for (int r = 0; r < csize; ++r) {
    kmin = min(kmin, peer(sh.minmax, r)[0]);
    kmax = max(kmax, peer(sh.minmax, r)[1]);
  }

  uint32_t need = (uint32_t)(n - first - last);  // places left for the middle's values
  // The bin searched: keys lo .. lo + span (inclusive).  Ends with a
  // threshold: values above it are taken, of those equal to it the first
  // `need` (need 0: none, or none left to take).
  uint32_t lo = kmin, span = kmax - kmin, above = 0xffffffffu;  // taken: key > above
  bool ties = false;
  if (need > 0) {
    for (int pass = 0;; ++pass) {
      const int bits = 32 - __clz(span);
      const int shift = bits > kSelBinBits ? bits - kSelBinBits : 0;
      uint32_t* hist = sh.hist[pass & 1];
      each([&](int i, uint32_t k, bool in) {
        const uint32_t off = k - lo;
        in = in && i >= m0 && i < m1 && off <= span;
        // a warp whose values all share a bin (equal values do) counts once
        const uint32_t bin = in ? off >> shift : kSelBins;
        int same;
        __match_all_sync(0xffffffffu, bin, &same);
        if (in && (!same || lane == 0)) atomicAdd(hist + bin, same ? 32u : 1u);
      });
      cluster_sync();
      // from the top bin down: thread t takes the per = kSelBins / T bins
      // below kSelBins - t * per (T divides kSelBins)
      const int per = kSelBins / T;
      uint32_t sum = 0;
      for (int j = 0; j < per; ++j) {
        const int b = kSelBins - 1 - tid * per - j;
        for (int r = 0; r < csize; ++r) sum += peer(hist, r)[b];
      }
      uint32_t total;
      uint32_t before = select_block_scan(sum, sh.warp_a, total);
      if (before < need && need <= before + sum) {
        for (int j = 0; j < per; ++j) {
          const int b = kSelBins - 1 - tid * per - j;
          uint32_t c = 0;
          for (int r = 0; r < csize; ++r) c += peer(hist, r)[b];
          if (before + c >= need) {
            sh.found[0] = (uint32_t)b;
            sh.found[1] = before;
            sh.found[2] = c;
            break;
          }
          before += c;
        }
      }
      // the other histogram is cleared for the next pass: its readers were
      // past it two barriers ago
      if (pass > 0)
        for (int b = tid; b < kSelBins; b += T) sh.hist[(pass + 1) & 1][b] = 0u;
      cluster_sync();
      const uint32_t bin = sh.found[0];
      need -= sh.found[1];
      lo += bin << shift;
      span = min(span - (bin << shift), (1u << shift) - 1u);
      if (sh.found[2] == need) {  // the whole bin
        above = lo - 1u;  // lo = 0 (NaN keys): taken by the ties rule below
        need = 0;
        if (lo == 0u) {
          above = 0u;
          ties = true;
          need = 0xffffffffu;
        }
        break;
      }
      if (shift == 0) {  // one key: its first `need` values by index
        above = lo;
        ties = true;
        break;
      }
    }
  }

  // Place the taken values in index order: rounds of kSelRegs values a
  // thread; in a round, value u of warp w comes after every value of earlier
  // (u, w).  A taken value's place is the number of values before it that are
  // above the threshold (or at a forced index) plus the ties before it, up to
  // need.
  auto is_above = [&](int i, uint32_t k) { return i < m0 || i >= m1 || k > above; };
  auto is_tie = [&](int i, uint32_t k) { return ties && i >= m0 && i < m1 && k == above; };
  uint32_t base_above = 0, base_tie = 0;
  if (csize > 1) {
    uint32_t a = 0, e = 0;
    each([&](int i, uint32_t k, bool in) {
      if (in && is_above(i, k)) ++a;
      else if (in && is_tie(i, k)) ++e;
    });
    a = __reduce_add_sync(0xffffffffu, a);
    e = __reduce_add_sync(0xffffffffu, e);
    if (lane == 0) {
      sh.warp_a[wid] = a;
      sh.warp_b[wid] = e;
    }
    __syncthreads();
    if (wid == 0) {
      a = __reduce_add_sync(0xffffffffu, lane < nw ? sh.warp_a[lane] : 0u);
      e = __reduce_add_sync(0xffffffffu, lane < nw ? sh.warp_b[lane] : 0u);
      if (lane == 0) {
        sh.totals[0] = a;
        sh.totals[1] = e;
      }
    }
    cluster_sync();
    for (int r = 0; r < rank; ++r) {
      base_above += peer(sh.totals, r)[0];
      base_tie += peer(sh.totals, r)[1];
    }
  }
  auto round = [&](int r0, auto key_of) {
#pragma unroll
    for (int u = 0; u < kSelRegs; ++u) {
      const int i = r0 + u * T + tid;
      const bool in = i < i1;
      const uint32_t k = key_of(u, i);
      const uint32_t ba = __ballot_sync(0xffffffffu, in && is_above(i, k));
      const uint32_t be = __ballot_sync(0xffffffffu, in && is_tie(i, k));
      if (lane == 0) sh.counts[u][wid] = (uint32_t)__popc(ba) | ((uint32_t)__popc(be) << 16);
    }
    __syncthreads();
    // exclusive scan of the (u, warp) counts: at most 512 entries of at most
    // 32 each, so both halves of the packed sums stay below 2^16
    const int entries = kSelRegs * nw;
    const uint32_t c = tid < entries ? sh.counts[tid / nw][tid % nw] : 0u;
    uint32_t total;
    const uint32_t off = select_block_scan(c, sh.warp_a, total);
    if (tid < entries) sh.counts[tid / nw][tid % nw] = off;
    __syncthreads();
#pragma unroll
    for (int u = 0; u < kSelRegs; ++u) {
      const int i = r0 + u * T + tid;
      const bool in = i < i1;
      const uint32_t k = key_of(u, i);
      const bool fa = in && is_above(i, k), fe = in && is_tie(i, k);
      const uint32_t ba = __ballot_sync(0xffffffffu, fa), be = __ballot_sync(0xffffffffu, fe);
      const uint32_t o = sh.counts[u][wid], below = (1u << lane) - 1u;
      const uint32_t pa = base_above + (o & 0xffffu) + (uint32_t)__popc(ba & below);
      const uint32_t pe = base_tie + (o >> 16) + (uint32_t)__popc(be & below);
      if (fa || (fe && pe < need)) emit((int)(pa + min(pe, need)), i);
    }
    base_above += total & 0xffffu;
    base_tie += total >> 16;
    __syncthreads();  // counts are rewritten by the next round
  };
  round(i0, [&](int u, int) { return reg[u]; });
  for (int r0 = i0 + kSelRegs * T; r0 < i1; r0 += kSelRegs * T)
    round(r0, [&](int, int i) { return i < i1 ? select_key(value(i)) : 0u; });
  if (csize > 1) cg::this_cluster().sync();  // peers may still read this CTA's totals
}

// Threads per CTA and CTAs per row for rows of up to cap values.
struct SelectShape {
  int threads, cluster;
};
SelectShape select_shape(int64_t rows, int64_t cap);
// Launch of a kernel of `rows` clusters; dependent: a programmatic dependent
// of the stream's previous kernel.
cudaError_t launch_rows(const void* kernel, int64_t rows, const SelectShape& s, void** args,
                        bool dependent, cudaStream_t st);

}  // namespace tl
