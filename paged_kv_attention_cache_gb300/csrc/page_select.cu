// Bounds of the pages' keys, and the pages a decode step's query selects by
// them: what tl_paged_attn_decode_pages then reads instead of a sequence's
// whole history.
//
// Mathematics.  For a page and KV head, M_d and m_d are the largest and
// smallest live key value of channel d.  Any key k of the page has
// <q, k> <= sum_d max(q_d M_d, q_d m_d), so the sum ranks pages by the
// largest score a key of theirs could reach.  It is held in int8: codes of
// (M, m) with one f32 scale per (page, head), and of q with one scale per
// query head.  The sum is then a sum of whole numbers, below 2^24, with two
// f32 products after it, so a page's score, and with it the selection, is the
// same bit for bit however the work is split, at an eighth of the bytes of
// one bf16 key page of 16.
#include <algorithm>

#include "common.cuh"
#include "row_select.cuh"

namespace tl {

// A row of one of the two phases reads 16 bytes per lane.
enum PoolKind { kBf16 = 0, kF32 = 1, kE4m3 = 2, kInt8 = 3 };

template <int KIND>
struct PoolElem {
  static constexpr int kBytes = KIND == kF32 ? 4 : KIND == kBf16 ? 2 : 1;
  static constexpr int kPerVec = 16 / kBytes;
};

// 16 bytes of a pool row as floats (int8: times the row's scale, one rounding).
template <int KIND>
TL_DEVINLINE void widen_vec(const uint4& x, float scale, float* f) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (KIND == kF32) {
      f[i] = __uint_as_float(w[i]);
    } else if (KIND == kBf16) {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    } else if (KIND == kE4m3) {
      uint32_t lo, hi;
      asm("{\n .reg .b16 l, h;\n mov.b32 {l, h}, %2;\n cvt.rn.f16x2.e4m3x2 %0, l;\n"
          " cvt.rn.f16x2.e4m3x2 %1, h;\n}\n"
          : "=r"(lo), "=r"(hi)
          : "r"(w[i]));
#pragma unroll
      for (int h = 0; h < 2; ++h)
        asm("{\n .reg .b16 l, h;\n mov.b32 {l, h}, %2;\n cvt.f32.f16 %0, l;\n cvt.f32.f16 %1, h;\n}\n"
            : "=f"(f[4 * i + 2 * h]), "=f"(f[4 * i + 2 * h + 1])
            : "r"(h ? hi : lo));
    } else {
#pragma unroll
      for (int b = 0; b < 4; ++b)
        f[4 * i + b] = __fmul_rn((float)(int8_t)(w[i] >> (8 * b)), scale);
    }
  }
}

// max / min that return NaN when either is
TL_DEVINLINE float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;\n" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
TL_DEVINLINE float min_nan(float a, float b) {
  float r;
  asm("min.NaN.f32 %0, %1, %2;\n" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

struct BoundsParams {
  const void* k;
  const float* k_scales;  // int8 pools: [num_pages][h_kv][page_size]
  const int32_t* block_table;
  const int32_t* first_new;  // null: every block
  const int32_t* context_lens;
  int8_t* bounds;  // [num_pages][h_kv][2][d]: max codes, min codes
  float* scales;   // [num_pages][h_kv]
  int32_t max_pages_per_seq, B, h_kv, num_pages, page_size;
  uint32_t* error_word;
};

// One warp per (page, KV head), 32 / (lanes per row) keys at a time and up to
// 8 such loads in flight per lane.
template <int D, int KIND>
TL_DEVINLINE void page_bounds(const BoundsParams& P, int page, int g, int live, int lane) {
  using E = PoolElem<KIND>;
  constexpr int V = E::kPerVec, LPR = D / V, RPW = 32 / LPR, U = 8;
  const int col = lane % LPR, row = lane / LPR;
  const size_t stride = (size_t)P.h_kv * D * E::kBytes;  // bytes between a head's rows
  const unsigned char* base = static_cast<const unsigned char*>(P.k) +
                              (size_t)page * P.page_size * stride + (size_t)g * D * E::kBytes +
                              col * 16;
  const float* ks = KIND == kInt8 ? P.k_scales + ((size_t)page * P.h_kv + g) * P.page_size : nullptr;
  float top[V], low[V];
  // clean: the values as they are; otherwise a non-finite one counts as 0
  auto reduce = [&](bool clean) {
#pragma unroll
    for (int e = 0; e < V; ++e) {
      top[e] = -INFINITY;
      low[e] = INFINITY;
    }
    for (int r0 = 0; r0 < live; r0 += RPW * U) {
      uint4 x[U];
      float sc[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int r = min(r0 + u * RPW + row, live - 1);  // a repeated row changes nothing
        x[u] = __ldg(reinterpret_cast<const uint4*>(base + (size_t)r * stride));
        sc[u] = KIND == kInt8 ? __ldg(ks + r) : 0.f;
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        float f[V];
        widen_vec<KIND>(x[u], sc[u], f);
#pragma unroll
        for (int e = 0; e < V; ++e) {
          const float v = clean || fabsf(f[e]) <= 3.402823466e38f ? f[e] : 0.f;
          top[e] = max_nan(top[e], v);
          low[e] = min_nan(low[e], v);
        }
      }
    }
#pragma unroll
    for (int o = LPR; o < 32; o <<= 1)
#pragma unroll
      for (int e = 0; e < V; ++e) {
        top[e] = max_nan(top[e], __shfl_xor_sync(0xffffffffu, top[e], o));
        low[e] = min_nan(low[e], __shfl_xor_sync(0xffffffffu, low[e], o));
      }
    float m = 0.f;
#pragma unroll
    for (int e = 0; e < V; ++e) m = max_nan(m, max_nan(fabsf(top[e]), fabsf(low[e])));
#pragma unroll
    for (int o = 1; o < LPR; o <<= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
    return m;
  };
  float m = reduce(true);
  if (!(m <= 3.402823466e38f)) {  // a NaN or an infinity among the live keys
    if (lane == 0) report(P.error_word, TL_DEVERR_VALUE_RANGE);
    m = reduce(false);
  }
  const float s = __fdiv_rn(m, 127.f);
  if (row < 2) {  // the first row group writes the max codes, the second the min codes
    uint32_t packed[(V + 3) / 4];
#pragma unroll
    for (int e = 0; e < V; ++e) {
      const float b = row == 0 ? top[e] : low[e];
      const float c = s > 0.f ? fminf(fmaxf(rintf(__fdiv_rn(b, s)), -127.f), 127.f) : 0.f;
      const uint32_t byte = (uint32_t)(uint8_t)(int8_t)__float2int_rn(c);
      if (e % 4 == 0) packed[e / 4] = byte;
      else packed[e / 4] |= byte << (8 * (e % 4));
    }
    uint32_t* dst = reinterpret_cast<uint32_t*>(
        P.bounds + (((size_t)page * P.h_kv + g) * 2 + row) * D + col * V);
#pragma unroll
    for (int i = 0; i < V / 4; ++i) dst[i] = packed[i];
    if (RPW == 1) {  // an f32 row of 128 takes the whole warp: it writes both
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const float c = s > 0.f ? fminf(fmaxf(rintf(__fdiv_rn(low[e], s)), -127.f), 127.f) : 0.f;
        const uint32_t byte = (uint32_t)(uint8_t)(int8_t)__float2int_rn(c);
        if (e % 4 == 0) packed[e / 4] = byte;
        else packed[e / 4] |= byte << (8 * (e % 4));
      }
#pragma unroll
      for (int i = 0; i < V / 4; ++i) dst[D / 4 + i] = packed[i];
    }
    if (lane == 0) P.scales[(size_t)page * P.h_kv + g] = s;
  }
}

constexpr int kBoundsThreads = 256;
constexpr int kBoundsSeqs = 1024;  // sequences placed per round

// Blocks first_new / page_size .. (L - 1) / page_size of every sequence,
// times the heads, spread over the grid's warps: each CTA scans the
// sequences' block counts into shared memory, and a warp finds the sequence
// of its next (block, head) by a binary search.  The batch may be ragged (a
// prompt among decode steps): the work is even whatever the lengths, and the
// host needs to know none of them.
template <int D, int KIND>
__global__ void __launch_bounds__(kBoundsThreads) page_bounds_kernel(BoundsParams P) {
  __shared__ int start[kBoundsSeqs + 1];  // first block of each sequence of the round
  __shared__ uint32_t tmp[32];
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = blockIdx.x * (kBoundsThreads / 32) + (tid >> 5);
  const int nwarps = gridDim.x * (kBoundsThreads / 32);
  constexpr int PER = kBoundsSeqs / kBoundsThreads;
  for (int base = 0; base < P.B; base += kBoundsSeqs) {
    uint32_t n[PER], sum = 0;
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      const int b = base + tid * PER + j;
      n[j] = 0;
      if (b < P.B) {
        const int L = P.context_lens[b];
        const int f = P.first_new ? max(P.first_new[b], 0) : 0;
        if ((int64_t)L > (int64_t)P.max_pages_per_seq * P.page_size) {
          if (blockIdx.x == 0) report(P.error_word, TL_DEVERR_CONTEXT_RANGE);
        } else if (L > f) {
          n[j] = (uint32_t)((L - 1) / P.page_size - f / P.page_size + 1);
        }
      }
      sum += n[j];
    }
    uint32_t total;
    uint32_t at = select_block_scan(sum, tmp, total);
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      start[tid * PER + j] = (int)at;
      at += n[j];
    }
    if (tid == 0) start[kBoundsSeqs] = (int)total;
    __syncthreads();
    for (int64_t t = warp; t < (int64_t)total * P.h_kv; t += nwarps) {
      const int i = (int)(t / P.h_kv), g = (int)(t % P.h_kv);
      int lo = 0, hi = kBoundsSeqs;  // the last sequence that starts at or before i
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (start[mid] <= i) lo = mid;
        else hi = mid;
      }
      // sequences without blocks start where the next one does: the last of
      // equal starts is the one that has them
      const int b = base + lo;
      const int f = P.first_new ? max(P.first_new[b], 0) : 0;
      const int blk = f / P.page_size + (i - start[lo]);
      const int live = min(P.page_size, P.context_lens[b] - blk * P.page_size);
      const int page = __ldg(P.block_table + (size_t)b * P.max_pages_per_seq + blk);
      if (page < 0 || page >= P.num_pages) {
        if (lane == 0) report(P.error_word, TL_DEVERR_PAGE_RANGE);
        continue;
      }
      page_bounds<D, KIND>(P, page, g, live, lane);
    }
    __syncthreads();  // start is rewritten by the next round
  }
}

// ------------------------------------------------------------------ scores --

struct ScoreParams {
  const void* q;  // [B][h_q][d], bf16 or f32
  const int8_t* bounds;
  const float* scales;
  const int32_t* block_table;
  const int32_t* context_lens;
  float* scores;  // [B][h_kv][max_pages_per_seq]
  int32_t max_pages_per_seq, B, h_q, h_kv, group, num_pages, page_size;
  uint32_t* error_word;
};

constexpr int kScoreWarps = 8;
constexpr int kScoreTile = 128;  // pages of a CTA

__host__ __device__ inline int score_heads(int h_kv) { return h_kv < kScoreWarps ? h_kv : kScoreWarps; }

// Blocks a sequence has, or 0 when its length is past its table.
TL_DEVINLINE int blocks_of(int L, int max_pages, int page_size) {
  return L <= 0 || (int64_t)L > (int64_t)max_pages * page_size ? 0 : (L - 1) / page_size + 1;
}

// Scores of a tile of a sequence's pages.  A CTA quantises the query rows of
// its heads once; its warps each take one head and walk the tile's pages, D/16
// lanes to a page (16 max codes and 16 min codes a lane), neighbouring warps
// on neighbouring heads of the same page, whose codes are one run of memory.
template <int D, int G, bool QF32>
__global__ void __launch_bounds__(kScoreWarps * 32) page_score_kernel(ScoreParams P) {
  constexpr int LP = D / 16, PW = 32 / LP, U = 4;  // lanes a page, pages a load, loads in flight
  __shared__ __align__(16) int8_t q_codes[kScoreWarps * G][D];
  __shared__ float q_scale[kScoreWarps * G];
  const int b = blockIdx.z, lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int L = P.context_lens[b];
  const int nb = blocks_of(L, P.max_pages_per_seq, P.page_size);
  const int p0 = blockIdx.x * kScoreTile, p1 = min(p0 + kScoreTile, nb);
  if (p0 >= p1) return;
  const int hs = score_heads(P.h_kv), g0 = blockIdx.y * hs, heads = min(hs, P.h_kv - g0);
  // query rows: code = rint(q / t) clamped to +-127, t = max|q| / 127
  for (int r = w; r < heads * P.group; r += kScoreWarps) {
    const size_t row = ((size_t)b * P.h_q + (size_t)g0 * P.group + r) * D;
    float x[D / 32], m = 0.f;
    bool bad = false;
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
      const size_t e = row + lane + 32 * i;
      x[i] = QF32 ? __ldg(static_cast<const float*>(P.q) + e)
                  : __uint_as_float((uint32_t)__ldg(static_cast<const unsigned short*>(P.q) + e) << 16);
      if (!isfinite(x[i])) {  // counts as 0
        bad = true;
        x[i] = 0.f;
      }
      m = fmaxf(m, fabsf(x[i]));
    }
    m = warp_max(m);
    const float t = __fdiv_rn(m, 127.f);
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
      const float c = t > 0.f ? fminf(fmaxf(rintf(__fdiv_rn(x[i], t)), -127.f), 127.f) : 0.f;
      q_codes[r][lane + 32 * i] = (int8_t)__float2int_rn(c);
    }
    if (lane == 0) q_scale[r] = t;
    if (__any_sync(0xffffffffu, bad) && lane == 0) report(P.error_word, TL_DEVERR_VALUE_RANGE);
  }
  __syncthreads();
  const int per_head = kScoreWarps / hs;  // warps that share a head
  if (w >= hs * per_head) return;
  const int gi = w % hs, sub = w / hs, g = g0 + gi;
  if (gi >= heads) return;
  const int col = lane % LP, row = lane / LP;
  // the query codes of this lane's 16 channels, split by sign
  uint32_t qp[G][4], qn[G][4];
  float t[G];
#pragma unroll
  for (int r = 0; r < G; ++r) {
    t[r] = r < P.group ? q_scale[gi * P.group + r] : 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t c =
          r < P.group ? *reinterpret_cast<const uint32_t*>(&q_codes[gi * P.group + r][col * 16 + 4 * i])
                      : 0u;
      const uint32_t neg = __vcmplts4(c, 0u);  // 0xff in the bytes below 0
      qp[r][i] = c & ~neg;
      qn[r][i] = c & neg;
    }
  }
  float* out = P.scores + ((size_t)b * P.h_kv + g) * P.max_pages_per_seq;
  const int32_t* table = P.block_table + (size_t)b * P.max_pages_per_seq;
  for (int q0 = p0 + sub * PW * U; q0 < p1; q0 += per_head * PW * U) {
    uint4 mx[U], mn[U];
    float sc[U];
    bool ok[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = q0 + u * PW + row;
      const int page = i < p1 ? __ldg(table + i) : -1;
      ok[u] = page >= 0 && page < P.num_pages;
      if (i < p1 && !ok[u] && col == 0) report(P.error_word, TL_DEVERR_PAGE_RANGE);
      const size_t at = (size_t)(ok[u] ? page : 0) * P.h_kv + g;
      const uint4* src = reinterpret_cast<const uint4*>(P.bounds + at * 2 * D) + col;
      mx[u] = __ldg(src);
      mn[u] = __ldg(src + LP);
      sc[u] = __ldg(P.scales + at);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const uint32_t a[4] = {mx[u].x, mx[u].y, mx[u].z, mx[u].w};
      const uint32_t c[4] = {mn[u].x, mn[u].y, mn[u].z, mn[u].w};
      float best = -INFINITY;
#pragma unroll
      for (int r = 0; r < G; ++r) {
        if (r >= P.group) break;  // groups between two instantiations (5 runs the form of 8)
        int dot = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          dot = __dp4a((int)qp[r][i], (int)a[i], dot);
          dot = __dp4a((int)qn[r][i], (int)c[i], dot);
        }
#pragma unroll
        for (int o = 1; o < LP; o <<= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
        // a whole number below 2^24: exact as a float
        best = fmaxf(best, __fmul_rn(__fmul_rn((float)dot, sc[u]), t[r]));
      }
      const int i = q0 + u * PW + row;
      if (i < p1 && col == 0) out[i] = ok[u] ? best : -INFINITY;
    }
  }
}

// ------------------------------------------------------------------ select --

struct PageSelectParams {
  const float* scores;
  const int32_t* block_table;
  const int32_t* context_lens;
  int32_t* table;  // [B][h_kv][n]
  int32_t* lens;   // [B]
  int32_t max_pages_per_seq, h_kv, page_size, n, first, last;
  uint32_t* error_word;
};

__global__ void __launch_bounds__(kSelMaxThreads) page_select_kernel(PageSelectParams P, int csize) {
  __shared__ SelectShared sh;
  asm volatile("griddepcontrol.wait;\n" ::: "memory");
  const int row = blockIdx.x / csize, rank = blockIdx.x % csize;
  const int b = row / P.h_kv;
  const int L = P.context_lens[b];
  const int nb = blocks_of(L, P.max_pages_per_seq, P.page_size);
  if (row % P.h_kv == 0 && rank == 0 && threadIdx.x == 0) {
    P.lens[b] = nb == 0 ? 0 : nb <= P.n ? L : (P.n - 1) * P.page_size + (L - 1) % P.page_size + 1;
    if (nb == 0 && L > 0) report(P.error_word, TL_DEVERR_CONTEXT_RANGE);
  }
  const float* x = P.scores + (size_t)row * P.max_pages_per_seq;
  const int32_t* from = P.block_table + (size_t)b * P.max_pages_per_seq;
  int32_t* to = P.table + (size_t)row * P.n;
  select_row(
      sh, nb, P.n, P.first, P.last, rank, csize, [&](int i) { return __ldcg(x + i); },
      [&](int pos, int i) { to[pos] = __ldg(from + i); }, [&](int pos) { to[pos] = -1; });
}

}  // namespace tl

// -------------------------------------------------------------------- host --

namespace tl {

static tl_status bounds_impl(const void* k, const float* k_scales, const int32_t* block_table,
                             int32_t max_pages_per_seq, const int32_t* first_new,
                             const int32_t* context_lens, int8_t* bounds, float* bound_scales,
                             int32_t B, int32_t h_kv, int32_t d, int32_t num_pages,
                             int32_t page_size, int kind, uint32_t* error_word, void* stream) {
  if (B <= 0 || h_kv <= 0 || d <= 0 || num_pages <= 0 || page_size <= 0 || max_pages_per_seq <= 0)
    return TL_ERR_INVALID_ARG;
  if (!k || !block_table || !context_lens || !bounds || !bound_scales) return TL_ERR_INVALID_ARG;
  if (!aligned16(k) || !aligned16(bounds) || !aligned16(bound_scales) || !aligned16(k_scales) ||
      (reinterpret_cast<uintptr_t>(block_table) & 3u) ||
      (reinterpret_cast<uintptr_t>(context_lens) & 3u) ||
      (reinterpret_cast<uintptr_t>(first_new) & 3u))
    return TL_ERR_INVALID_ARG;
  if ((d != 64 && d != 128) || page_size > 256 || kind < 0) return TL_ERR_UNSUPPORTED;
  if ((int64_t)num_pages * page_size >= ((int64_t)1 << 31)) return TL_ERR_UNSUPPORTED;
  // block counts are summed in 32 bits
  if ((int64_t)B * max_pages_per_seq > INT32_MAX) return TL_ERR_UNSUPPORTED;
  BoundsParams P;
  P.k = k;
  P.k_scales = k_scales;
  P.block_table = block_table;
  P.first_new = first_new;
  P.context_lens = context_lens;
  P.bounds = bounds;
  P.scales = bound_scales;
  P.max_pages_per_seq = max_pages_per_seq;
  P.B = B;
  P.h_kv = h_kv;
  P.num_pages = num_pages;
  P.page_size = page_size;
  P.error_word = error_word;
  const int64_t most = ((int64_t)B * max_pages_per_seq * h_kv + kBoundsThreads / 32 - 1) /
                       (kBoundsThreads / 32);
  const unsigned grid = (unsigned)std::min<int64_t>(most, (int64_t)num_sms() * 6);
  cudaStream_t st = (cudaStream_t)stream;
#define TL_BOUNDS(K)                                                              \
  do {                                                                            \
    if (d == 128) page_bounds_kernel<128, K><<<grid, kBoundsThreads, 0, st>>>(P); \
    else page_bounds_kernel<64, K><<<grid, kBoundsThreads, 0, st>>>(P);           \
  } while (0)
  if (kind == kBf16) TL_BOUNDS(kBf16);
  else if (kind == kF32) TL_BOUNDS(kF32);
  else if (kind == kE4m3) TL_BOUNDS(kE4m3);
  else TL_BOUNDS(kInt8);
#undef TL_BOUNDS
  return launch_status();
}

template <int D, bool QF32>
static void launch_score(const ScoreParams& P, dim3 grid, cudaStream_t st) {
  const int threads = kScoreWarps * 32;
  if (P.group <= 1) page_score_kernel<D, 1, QF32><<<grid, threads, 0, st>>>(P);
  else if (P.group <= 2) page_score_kernel<D, 2, QF32><<<grid, threads, 0, st>>>(P);
  else if (P.group <= 4) page_score_kernel<D, 4, QF32><<<grid, threads, 0, st>>>(P);
  else if (P.group <= 8) page_score_kernel<D, 8, QF32><<<grid, threads, 0, st>>>(P);
  else page_score_kernel<D, 16, QF32><<<grid, threads, 0, st>>>(P);
}

SelectShape select_shape(int64_t rows, int64_t cap) {
  SelectShape s;
  s.threads = cap <= 4096 ? 256 : cap <= 8192 ? 512 : kSelMaxThreads;
  s.cluster = 1;
  // more CTAs a row while the rows leave SMs empty and a slice stays long
  while (s.cluster < 8 && cap > (int64_t)4096 * s.cluster && rows * s.cluster * 2 <= num_sms())
    s.cluster *= 2;
  // a row past the registers of its CTAs is split further whatever the rows
  while (s.cluster < 8 && cap > (int64_t)kSelRegs * kSelMaxThreads * s.cluster) s.cluster *= 2;
  return s;
}

cudaError_t launch_rows(const void* kernel, int64_t rows, const SelectShape& s, void** args,
                        bool dependent, cudaStream_t st) {
  cudaLaunchAttribute attr[2];
  int n = 0;
  if (s.cluster > 1) {
    attr[n].id = cudaLaunchAttributeClusterDimension;
    attr[n].val.clusterDim.x = (unsigned)s.cluster;
    attr[n].val.clusterDim.y = 1;
    attr[n].val.clusterDim.z = 1;
    ++n;
  }
  if (dependent) {
    attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[n].val.programmaticStreamSerializationAllowed = 1;
    ++n;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(rows * s.cluster));
  cfg.blockDim = dim3((unsigned)s.threads);
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = (unsigned)n;
  return cudaLaunchKernelExC(&cfg, kernel, args);
}

}  // namespace tl

extern "C" tl_status tl_kv_page_bounds(const void* k_cache, const int32_t* block_table,
                                       int32_t max_pages_per_seq, const int32_t* first_new,
                                       const int32_t* context_lens, int8_t* bounds,
                                       float* bound_scales, int32_t B, int32_t h_kv, int32_t d,
                                       int32_t num_pages, int32_t page_size, tl_dtype dtype,
                                       uint32_t* error_word, void* stream) {
  const int kind = dtype == TL_BF16       ? tl::kBf16
                   : dtype == TL_F32      ? tl::kF32
                   : dtype == TL_FP8_E4M3 ? tl::kE4m3
                                          : -1;
  return tl::bounds_impl(k_cache, nullptr, block_table, max_pages_per_seq, first_new, context_lens,
                         bounds, bound_scales, B, h_kv, d, num_pages, page_size, kind, error_word,
                         stream);
}

extern "C" tl_status tl_kv_page_bounds_int8(const int8_t* k_codes, const float* k_scales,
                                            const int32_t* block_table, int32_t max_pages_per_seq,
                                            const int32_t* first_new, const int32_t* context_lens,
                                            int8_t* bounds, float* bound_scales, int32_t B,
                                            int32_t h_kv, int32_t d, int32_t num_pages,
                                            int32_t page_size, uint32_t* error_word,
                                            void* stream) {
  if (!k_scales) return TL_ERR_INVALID_ARG;
  return tl::bounds_impl(k_codes, k_scales, block_table, max_pages_per_seq, first_new,
                         context_lens, bounds, bound_scales, B, h_kv, d, num_pages, page_size,
                         tl::kInt8, error_word, stream);
}

extern "C" size_t tl_kv_page_select_workspace_size(int32_t B, int32_t h_kv,
                                                   int32_t max_pages_per_seq) {
  if (B <= 0 || h_kv <= 0 || max_pages_per_seq <= 0) return 0;
  return tl::align_up(sizeof(float) * (size_t)B * h_kv * max_pages_per_seq, 256);
}

extern "C" tl_status tl_kv_page_select(const void* q, tl_dtype q_dtype, const int8_t* bounds,
                                       const float* bound_scales, const int32_t* block_table,
                                       int32_t max_pages_per_seq, const int32_t* context_lens,
                                       int32_t n_select, int32_t keep_first, int32_t keep_last,
                                       int32_t* page_table, int32_t* page_lens, int32_t B,
                                       int32_t h_q, int32_t h_kv, int32_t d, int32_t num_pages,
                                       int32_t page_size, void* workspace, size_t workspace_bytes,
                                       uint32_t* error_word, void* stream) {
  using namespace tl;
  if (B <= 0 || h_q <= 0 || h_kv <= 0 || d <= 0 || num_pages <= 0 || page_size <= 0 ||
      max_pages_per_seq <= 0 || n_select <= 0 || keep_first < 0 || keep_last < 1 ||
      (int64_t)keep_first + keep_last > n_select || h_q % h_kv)
    return TL_ERR_INVALID_ARG;
  if (!q || !bounds || !bound_scales || !block_table || !context_lens || !page_table || !page_lens)
    return TL_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(bounds) || !aligned16(bound_scales) || !aligned16(page_table) ||
      !aligned16(page_lens) || (reinterpret_cast<uintptr_t>(block_table) & 3u) ||
      (reinterpret_cast<uintptr_t>(context_lens) & 3u))
    return TL_ERR_INVALID_ARG;
  if (q_dtype != TL_BF16 && q_dtype != TL_F32) return TL_ERR_UNSUPPORTED;
  if ((d != 64 && d != 128) || h_q / h_kv > 16 || page_size > 256 || B > 65535 ||
      (int64_t)num_pages * page_size >= ((int64_t)1 << 31) ||
      (int64_t)n_select * page_size >= ((int64_t)1 << 31) ||
      (int64_t)B * h_kv > INT32_MAX / 8 || (h_kv + kScoreWarps - 1) / kScoreWarps > 65535)
    return TL_ERR_UNSUPPORTED;
  if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u) ||
      workspace_bytes < tl_kv_page_select_workspace_size(B, h_kv, max_pages_per_seq))
    return TL_ERR_WORKSPACE;
  cudaStream_t st = (cudaStream_t)stream;
  ScoreParams S;
  S.q = q;
  S.bounds = bounds;
  S.scales = bound_scales;
  S.block_table = block_table;
  S.context_lens = context_lens;
  S.scores = static_cast<float*>(workspace);
  S.max_pages_per_seq = max_pages_per_seq;
  S.B = B;
  S.h_q = h_q;
  S.h_kv = h_kv;
  S.group = h_q / h_kv;
  S.num_pages = num_pages;
  S.page_size = page_size;
  S.error_word = error_word;
  const int hs = score_heads(h_kv);
  const dim3 grid((unsigned)((max_pages_per_seq + kScoreTile - 1) / kScoreTile),
                  (unsigned)((h_kv + hs - 1) / hs), (unsigned)B);
  if (d == 128) {
    if (q_dtype == TL_F32) launch_score<128, true>(S, grid, st);
    else launch_score<128, false>(S, grid, st);
  } else {
    if (q_dtype == TL_F32) launch_score<64, true>(S, grid, st);
    else launch_score<64, false>(S, grid, st);
  }
  if (launch_status() != TL_OK) return TL_ERR_CUDA;
  PageSelectParams P;
  P.scores = S.scores;
  P.block_table = block_table;
  P.context_lens = context_lens;
  P.table = page_table;
  P.lens = page_lens;
  P.max_pages_per_seq = max_pages_per_seq;
  P.h_kv = h_kv;
  P.page_size = page_size;
  P.n = n_select;
  P.first = keep_first;
  P.last = keep_last;
  P.error_word = error_word;
  const int64_t rows = (int64_t)B * h_kv;
  const SelectShape s = select_shape(rows, max_pages_per_seq);
  int csize = s.cluster;
  void* args[] = {&P, &csize};
  if (launch_rows(reinterpret_cast<const void*>(page_select_kernel), rows, s, args, true, st) !=
      cudaSuccess)
    return TL_ERR_CUDA;
  return launch_status();
}
