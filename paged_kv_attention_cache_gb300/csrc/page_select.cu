// Bounds of the pages' keys, and the pages a decode step's query selects by
// them: what tl_paged_attn_decode_pages then reads instead of a sequence's
// whole history.
//
// Mathematics.  For a page and KV head, M_d and m_d are the largest and
// smallest live key value of channel d.  Any key k of the page has
// <q, k> <= sum_d max(q_d M_d, q_d m_d), so the sum ranks pages by the
// largest score a key of theirs could reach (page selection by per-channel
// minima and maxima: Tang et al., "Quest: Query-Aware Sparsity for Efficient
// Long-Context LLM Inference", 2024).  It is estimated in int8: codes of (M, m)
// with one f32 scale per (page, head), and of q with one scale per query head,
// all rounded to nearest (so the estimate may lie below the sum).  It is then a
// sum of whole numbers, below 2^24, with two f32 products after it, so a page's
// score, and with it the selection, is the same bit for bit however the work is
// split, at a sixteenth of the bytes of the page's keys (16 of bf16; an eighth
// of one-byte ones).
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

// D(16x8, s32) += A(16x32, s8, row) * B(32x8, s8, col)
TL_DEVINLINE void mma_s8_16832(int* c, const uint32_t* a, const uint32_t* b) {
  asm("mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};\n"
      : "+r"(c[0]), "+r"(c[1]), "+r"(c[2]), "+r"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
}

// round-half-even(x / s) as the f32 quotient rounds, clamped to +-127, for s >
// 0 and |x / s| <= 128: __fdividef is documented within 2 ulp (2^-22 of the
// value) and the product adds half a one, 3 x 10^-7 together, so x * (1 / s) is
// within 4 x 10^-5 of the quotient; it rounds alike unless it lies within 5 x
// 10^-4 of a half, where (and for an s whose reciprocal is out of range) the
// division is done.
struct Quotient {
  float s, inv;
  bool fast;
  TL_DEVINLINE explicit Quotient(float scale) : s(scale), inv(0.f), fast(scale > 1e-30f && scale < 1e30f) {
    if (fast) inv = __fdividef(1.f, s);
  }
  TL_DEVINLINE int code(float x) const {
    const float r = x * inv;
    float c = rintf(r);
    if (!fast || fabsf(r - c) > 0.4995f) c = s > 0.f ? rintf(__fdiv_rn(x, s)) : 0.f;
    return __float2int_rn(fminf(fmaxf(c, -127.f), 127.f));
  }
};

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

// Running max and min of a lane's 16-byte vectors.  16-bit values go two at a
// time (a packed max and min per pair; e4m3 codes are fp16 values too); f32 and
// scaled int8 values one at a time.
template <int KIND>
struct Extremes {
  static constexpr int V = PoolElem<KIND>::kPerVec;
  static constexpr bool kPacked = KIND == kBf16 || KIND == kE4m3;
  static constexpr int N = kPacked ? V / 2 : V;
  uint32_t top[N], low[N];  // packed pairs, or f32 bits
  TL_DEVINLINE static uint32_t max_of(uint32_t a, uint32_t b) {
    if (KIND == kBf16) asm("max.NaN.bf16x2 %0, %0, %1;\n" : "+r"(a) : "r"(b));
    else if (KIND == kE4m3) asm("max.NaN.f16x2 %0, %0, %1;\n" : "+r"(a) : "r"(b));
    else return __float_as_uint(max_nan(__uint_as_float(a), __uint_as_float(b)));
    return a;
  }
  TL_DEVINLINE static uint32_t min_of(uint32_t a, uint32_t b) {
    if (KIND == kBf16) asm("min.NaN.bf16x2 %0, %0, %1;\n" : "+r"(a) : "r"(b));
    else if (KIND == kE4m3) asm("min.NaN.f16x2 %0, %0, %1;\n" : "+r"(a) : "r"(b));
    else return __float_as_uint(min_nan(__uint_as_float(a), __uint_as_float(b)));
    return a;
  }
  TL_DEVINLINE void clear() {  // -inf, +inf
    constexpr uint32_t inf = KIND == kBf16 ? 0x7f807f80u : KIND == kE4m3 ? 0x7c007c00u : 0x7f800000u;
    constexpr uint32_t sign = kPacked ? 0x80008000u : 0x80000000u;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      top[i] = inf | sign;
      low[i] = inf;
    }
  }
  TL_DEVINLINE void add(const uint4& x, float scale) {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
    uint32_t v[N];
    if constexpr (KIND == kBf16 || KIND == kF32) {
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = w[i];
    } else if constexpr (KIND == kE4m3) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        asm("{\n .reg .b16 l, h;\n mov.b32 {l, h}, %2;\n cvt.rn.f16x2.e4m3x2 %0, l;\n"
            " cvt.rn.f16x2.e4m3x2 %1, h;\n}\n"
            : "=r"(v[2 * i]), "=r"(v[2 * i + 1])
            : "r"(w[i]));
    } else {
      float f[V];
      widen_vec<KIND>(x, scale, f);
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = __float_as_uint(f[i]);
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
      top[i] = max_of(top[i], v[i]);
      low[i] = min_of(low[i], v[i]);
    }
  }
  TL_DEVINLINE void fold(int o) {  // with the lane `o` away
#pragma unroll
    for (int i = 0; i < N; ++i) {
      top[i] = max_of(top[i], __shfl_xor_sync(0xffffffffu, top[i], o));
      low[i] = min_of(low[i], __shfl_xor_sync(0xffffffffu, low[i], o));
    }
  }
  TL_DEVINLINE static void floats(const uint32_t* x, float* f) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if (KIND == kBf16) {
        f[2 * i] = __uint_as_float(x[i] << 16);
        f[2 * i + 1] = __uint_as_float(x[i] & 0xffff0000u);
      } else if (KIND == kE4m3) {
        asm("{\n .reg .b16 l, h;\n mov.b32 {l, h}, %2;\n cvt.f32.f16 %0, l;\n cvt.f32.f16 %1, h;\n}\n"
            : "=f"(f[2 * i]), "=f"(f[2 * i + 1])
            : "r"(x[i]));
      } else {
        f[i] = __uint_as_float(x[i]);
      }
    }
  }
};

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
  auto largest = [&]() {  // of the magnitudes, over the whole row
    float m = 0.f;
#pragma unroll
    for (int e = 0; e < V; ++e) m = max_nan(m, max_nan(fabsf(top[e]), fabsf(low[e])));
#pragma unroll
    for (int o = 1; o < LPR; o <<= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
    return m;
  };
  Extremes<KIND> ext;
  ext.clear();
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
    for (int u = 0; u < U; ++u) ext.add(x[u], sc[u]);
  }
#pragma unroll
  for (int o = LPR; o < 32; o <<= 1) ext.fold(o);
  ext.floats(ext.top, top);
  ext.floats(ext.low, low);
  float m = largest();
  if (!(m <= 3.402823466e38f)) {  // a NaN or an infinity among the live keys: it counts as 0
    if (lane == 0) report(P.error_word, TL_DEVERR_VALUE_RANGE);
#pragma unroll
    for (int e = 0; e < V; ++e) {
      top[e] = -INFINITY;
      low[e] = INFINITY;
    }
    for (int r0 = 0; r0 < live; r0 += RPW) {
      const int r = min(r0 + row, live - 1);
      float f[V];
      widen_vec<KIND>(__ldg(reinterpret_cast<const uint4*>(base + (size_t)r * stride)),
                      KIND == kInt8 ? __ldg(ks + r) : 0.f, f);
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const float v = fabsf(f[e]) <= 3.402823466e38f ? f[e] : 0.f;
        top[e] = fmaxf(top[e], v);
        low[e] = fminf(low[e], v);
      }
    }
#pragma unroll
    for (int o = LPR; o < 32; o <<= 1)
#pragma unroll
      for (int e = 0; e < V; ++e) {
        top[e] = fmaxf(top[e], __shfl_xor_sync(0xffffffffu, top[e], o));
        low[e] = fminf(low[e], __shfl_xor_sync(0xffffffffu, low[e], o));
      }
    m = largest();
  }
  const float s = __fdiv_rn(m, 127.f);
  const Quotient quot(s);
  if (row < 2) {  // the first row group writes the max codes, the second the min codes
    uint32_t packed[(V + 3) / 4];
#pragma unroll
    for (int e = 0; e < V; ++e) {
      const float b = row == 0 ? top[e] : low[e];
      const uint32_t byte = (uint32_t)(uint8_t)(int8_t)quot.code(b);
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
        const uint32_t byte = (uint32_t)(uint8_t)(int8_t)quot.code(low[e]);
        if (e % 4 == 0) packed[e / 4] = byte;
        else packed[e / 4] |= byte << (8 * (e % 4));
      }
#pragma unroll
      for (int i = 0; i < V / 4; ++i) dst[D / 4 + i] = packed[i];
    }
    if (lane == 0) P.scales[(size_t)page * P.h_kv + g] = s;
  }
}

// The first of n things that share `i` of `shares` takes (the first n % shares
// shares take one more).
TL_DEVINLINE uint32_t even_share(uint32_t n, uint32_t i, uint32_t shares) {
  const uint32_t q = n / shares;
  return q * i + min(i, n - q * shares);
}

constexpr int kBoundsThreads = 256;
// CTAs an SM holds at once (one-byte vectors are 16 channels a lane: 80
// registers instead of 64).
__host__ __device__ constexpr int bounds_ctas(int kind) {
  return kind == kInt8 || kind == kE4m3 ? 3 : 4;
}
constexpr int kBoundsSeqs = 1024;  // sequences placed per round

// Blocks first_new / page_size .. (L - 1) / page_size of every sequence,
// times the heads, in even runs over the grid's warps: each CTA scans the
// sequences' block counts into shared memory, and a warp finds the sequence
// of its run by a binary search.  The batch may be ragged (a prompt among
// decode steps): the work is even whatever the lengths, and the host needs to
// know none of them.  One wave of CTAs, as many as an SM takes.  8 prompts of
// 6,144-8,192 keys (8 KV heads of 128) take 24.3 us in bf16 (125 MB, 5.1 TB/s)
// and 42.5 in f32 (242 MB, 5.7 TB/s), bound by HBM; 36.1 in e4m3 (66 MB) and
// 56.9 in int8 (68 MB), bound by the arithmetic: 16 conversions (int8: and
// products with the key's scale) a lane and 16 bytes.  With a CTA an SM more
// than fit, a second wave of a third, they took 41.0 and 67.3.  A decode step
// of 64 sequences, a page each, takes 4.8 us (bf16) to 7.0 (int8): a launch and
// three dependent reads.
template <int D, int KIND>
__global__ void __launch_bounds__(kBoundsThreads, bounds_ctas(KIND)) page_bounds_kernel(BoundsParams P) {
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
    uint32_t at = select_block_scan(sum, tmp, total);  // the loop's barriers free tmp
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      start[tid * PER + j] = (int)at;
      at += n[j];
    }
    if (tid == 0) start[kBoundsSeqs] = (int)total;
    __syncthreads();
    // this warp's run of (block, head) pairs, heads innermost: a page's heads
    // are one run of memory
    const uint32_t tasks = total * (uint32_t)P.h_kv;
    uint32_t t = even_share(tasks, (uint32_t)warp, (uint32_t)nwarps);
    const uint32_t t1 = even_share(tasks, (uint32_t)warp + 1, (uint32_t)nwarps);
    while (t < t1) {
      const int i = (int)(t / (uint32_t)P.h_kv);
      int lo = 0, hi = kBoundsSeqs;  // the last sequence that starts at or before block i
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (start[mid] <= i) lo = mid;
        else hi = mid;
      }
      // sequences without blocks start where the next one does: the last of
      // equal starts is the one that has them
      const int b = base + lo;
      const int f = P.first_new ? max(P.first_new[b], 0) : 0, L = P.context_lens[b];
      int g = (int)(t - (uint32_t)i * (uint32_t)P.h_kv);
      const int first = f / P.page_size + (i - start[lo]);
      const int n_blk = start[lo + 1] - i;  // of the sequence from here
      const int32_t* table = P.block_table + (size_t)b * P.max_pages_per_seq + first;
      int page = __ldg(table);
      for (int k = 0; k < n_blk && t < t1; ++k, g = 0) {
        const int next = k + 1 < n_blk ? __ldg(table + k + 1) : -1;
        const int live = min(P.page_size, L - (first + k) * P.page_size);
        const bool ok = page >= 0 && page < P.num_pages;
        if (!ok && lane == 0) report(P.error_word, TL_DEVERR_PAGE_RANGE);
        for (; g < P.h_kv && t < t1; ++g, ++t)
          if (ok) page_bounds<D, KIND>(P, page, g, live, lane);
        page = next;
      }
    }
    __syncthreads();  // start is rewritten by the next round
  }
}

// ------------------------------------------------------------------ scores --

struct ScoreParams {
  const void* q;  // [B][h_q][d], bf16 or f32
  int8_t* q_codes;  // [B][h_q][d]
  float* q_scales;  // [B][h_q]
  const int8_t* bounds;
  const float* scales;
  const int32_t* block_table;
  const int32_t* context_lens;
  float* scores;  // [B][h_kv][row_stride]
  int64_t row_stride;
  int32_t max_pages_per_seq, B, h_q, h_kv, group, num_pages, page_size;
  uint32_t* error_word;
};

// A row of scores starts on 16 bytes.
inline int64_t score_stride(int max_pages_per_seq) { return ((int64_t)max_pages_per_seq + 3) / 4 * 4; }

// Query rows as int8 codes, one warp a row: code = rint(q / t) clamped to
// +-127, t = max|q| / 127; a value that is not finite counts as 0.
template <int D, bool QF32>
__global__ void __launch_bounds__(256) page_query_kernel(ScoreParams P) {
  constexpr int E = D / 32;  // a lane's channels
  // the scores' kernel may start: it waits for these codes after its first copies
  asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
  const int lane = threadIdx.x & 31;
  const int64_t row = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  if (row >= (int64_t)P.B * P.h_q) return;
  float x[E];
  if (QF32) {
    const float* src = static_cast<const float*>(P.q) + row * D + lane * E;
#pragma unroll
    for (int i = 0; i < E; i += 2) *reinterpret_cast<float2*>(x + i) = __ldg(reinterpret_cast<const float2*>(src + i));
  } else {
    const uint32_t* src = reinterpret_cast<const uint32_t*>(
        static_cast<const unsigned short*>(P.q) + row * D + lane * E);
#pragma unroll
    for (int i = 0; i < E / 2; ++i) {
      const uint32_t w = __ldg(src + i);
      x[2 * i] = __uint_as_float(w << 16);
      x[2 * i + 1] = __uint_as_float(w & 0xffff0000u);
    }
  }
  bool bad = false;
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < E; ++i) {
    if (!isfinite(x[i])) {
      bad = true;
      x[i] = 0.f;
    }
    m = fmaxf(m, fabsf(x[i]));
  }
  m = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(m)));  // m >= 0
  const float t = __fdiv_rn(m, 127.f);
  const Quotient quot(t);
  uint32_t code = 0;
#pragma unroll
  for (int i = 0; i < E; ++i) code |= (uint32_t)(uint8_t)(int8_t)quot.code(x[i]) << (8 * i);
  int8_t* dst = P.q_codes + row * D + lane * E;
  if (E == 4) *reinterpret_cast<uint32_t*>(dst) = code;
  else *reinterpret_cast<uint16_t*>(dst) = (uint16_t)code;
  if (lane == 0) P.q_scales[row] = t;
  if (__any_sync(0xffffffffu, bad) && lane == 0) report(P.error_word, TL_DEVERR_VALUE_RANGE);
}

constexpr int kScoreWarps = 8;    // that compute; one more copies
constexpr int kScoreThreads = (kScoreWarps + 1) * 32;
constexpr int kScoreUnit = 4;     // pages; a CTA takes a run of units
constexpr int kScoreSeqs = 1024;  // sequences placed per round
constexpr int kScoreStages = 3;

// Heads a CTA scores (grid.y covers the others), and the warps that share one.
__host__ __device__ inline int score_heads(int h_kv) { return h_kv < kScoreWarps ? h_kv : kScoreWarps; }

// Shared memory of a stage: 16 pages per warp of a head, each page's codes of
// the CTA's heads (one run of the bounds pool) and 16 bytes more, so that the
// same 16 bytes of 8 pages fall on different banks.
__host__ __device__ inline int score_page_bytes(int heads, int d) { return heads * 2 * d + 16; }
__host__ __device__ inline int score_stage_bytes(int heads, int d) {
  return 16 * (kScoreWarps / heads) * score_page_bytes(heads, d);
}

// Blocks a sequence has, or 0 when its length is past its table.
TL_DEVINLINE int blocks_of(int L, int max_pages, int page_size) {
  return L <= 0 || (int64_t)L > (int64_t)max_pages * page_size ? 0 : (L - 1) / page_size + 1;
}

// Scores of every page of every sequence, two CTAs per SM.  Each takes an even
// share of the batch's pages as one run (a scan of the sequences' block
// counts places it: the host knows no length).  One warp looks the pages up
// and copies them: a page's codes of the CTA's heads are one run of memory
// (2 KiB at 8 heads of 128), one bulk copy into a ring of stages, on from one
// sequence's pages to the next's.  The other warps take a KV head each, with
// no barrier among them: 16 pages are the rows of an m16n8k32 over int8, the
// group's query heads its columns, the sum over the channels of max code x (q
// code >= 0) and min code x (q code < 0) its k steps, in whole numbers.
// Bound: HBM, and past 8 heads a group the int8 MMA.  With the query's kernel
// and the selection, 64 sequences of 1,024-32,768 keys (142 MB of codes, 8 KV
// heads of 128, 5 query heads each) take 39.2 us and one of 131,072 17.1 us.
// The same sums by fp16 MMAs (the codes widened by byte permutes, exact with
// two chains) take as long there and 20-25% longer at 16 query heads.
template <int D, int NT>
__global__ void __launch_bounds__(kScoreThreads, 2) page_score_kernel(ScoreParams P) {
  constexpr int KS = D / 32;  // k steps of the max codes, and of the min codes
  constexpr int NST = kScoreStages;
  extern __shared__ __align__(16) unsigned char score_sm[];
  __shared__ int start[kScoreSeqs + 1];  // first unit of each sequence of the round
  __shared__ uint32_t tmp[32];
  __shared__ unsigned long long full[NST], empty[NST];
  __shared__ int abort_flag;
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  const int hs = score_heads(P.h_kv), g0 = blockIdx.y * hs, heads = min(hs, P.h_kv - g0);
  const int per_head = kScoreWarps / hs;
  const int page_bytes = score_page_bytes(hs, D), stage_bytes = score_stage_bytes(hs, D);
  const int stage_pages = 16 * per_head;
  const uint32_t sm0 = smem_u32(score_sm);
  // the selection may take the SMs that this grid leaves (it waits for the
  // grid's end before it reads a score)
  asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
  if (tid == 0) {
    abort_flag = 0;
    for (int s = 0; s < NST; ++s) {
      mbar_init(smem_u32(&full[s]), 1);
      mbar_init(smem_u32(&empty[s]), (uint32_t)(heads * per_head));
    }
    fence_mbar_init();
  }
  int slot = 0;          // of the ring, in step in every warp
  uint32_t parity = 0;   // of the slot's phase
  uint32_t stages = 0;   // copied (the copying warp)
  auto advance = [&]() {
    slot = slot + 1 == NST ? 0 : slot + 1;
    parity ^= slot == 0 ? 1u : 0u;
  };
  bool stop = false, waited = false;
  for (int base = 0; base < P.B; base += kScoreSeqs) {
    constexpr int PER = (kScoreSeqs + kScoreThreads - 1) / kScoreThreads;
    uint32_t n[PER], sum = 0;
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      const int i = tid * PER + j, b = base + i;
      const int nb = i < kScoreSeqs && b < P.B
                         ? blocks_of(P.context_lens[b], P.max_pages_per_seq, P.page_size)
                         : 0;
      n[j] = (uint32_t)(nb + kScoreUnit - 1) / kScoreUnit;
      sum += n[j];
    }
    uint32_t total;
    // the previous round's start and tmp are read; a wait that gave up in any
    // warp ends the rounds for all
    if (__syncthreads_or(stop)) break;
    uint32_t at = select_block_scan(sum, tmp, total);
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      if (tid * PER + j < kScoreSeqs) start[tid * PER + j] = (int)at;
      at += n[j];
    }
    if (tid == 0) start[kScoreSeqs] = (int)total;
    __syncthreads();
    const int u1 = (int)even_share(total, blockIdx.x + 1, gridDim.x);
    // The CTA's units as segments, one sequence each: pages p0 .. p1 of
    // sequence b in steps of a stage.  The copying warp and the others walk
    // them at their own pace.
    struct Segment {
      int next, b, p0, p1, steps;  // next: the first unit behind it
      const int32_t* table;
    } seg;
    seg.next = (int)even_share(total, blockIdx.x, gridDim.x);
    auto open = [&]() {
      const int u = seg.next;
      if (u >= u1) return false;
      int lo = 0, hi = min(kScoreSeqs, P.B - base);  // the last sequence that starts at or before u
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (start[mid] <= u) lo = mid;
        else hi = mid;
      }
      seg.b = base + lo;
      seg.next = min(u1, start[lo + 1]);
      seg.p0 = (u - start[lo]) * kScoreUnit;
      seg.p1 = min((seg.next - start[lo]) * kScoreUnit,
                   blocks_of(P.context_lens[seg.b], P.max_pages_per_seq, P.page_size));
      seg.steps = (seg.p1 - seg.p0 + stage_pages - 1) / stage_pages;
      seg.table = P.block_table + (size_t)seg.b * P.max_pages_per_seq;
      return true;
    };
    if (w == kScoreWarps) {
      // ---------------------------------------------------------- copies
      const uint32_t copy_bytes = (uint32_t)heads * 2 * D;
      while (!stop && open()) {
        const int n_pages = seg.p1 - seg.p0;
        // 32 entries of the table at a time, the next ones on their way
        int ahead = lane < n_pages ? __ldg(seg.table + seg.p0 + lane) : -1;
        int window = -1, held = 0;
        for (int k = 0; k < seg.steps; ++k) {
          if (!mbar_wait(smem_u32(&empty[slot]), parity ^ 1u, &abort_flag)) {
            stop = true;
            break;
          }
          const int n_here = min(stage_pages, n_pages - k * stage_pages);
          uint32_t bytes = 0;
          for (int c0 = 0; c0 < n_here; c0 += 32) {  // this stage's pages, a lane each
            const int i = k * stage_pages + c0;      // of the segment
            if (i >= held) {
              window = ahead;
              held += 32;
              ahead = held + lane < n_pages ? __ldg(seg.table + seg.p0 + held + lane) : -1;
            }
            const int page = __shfl_sync(0xffffffffu, window, (i & 31) + lane);
            const bool inside = lane < min(n_here - c0, min(32, stage_pages));
            const bool ok = inside && page >= 0 && page < P.num_pages;
            if (inside && !ok) report(P.error_word, TL_DEVERR_PAGE_RANGE);
            bytes += (uint32_t)__popc(__ballot_sync(0xffffffffu, ok)) * copy_bytes;
#ifdef TL_TEST_STALL_FIRST_STAGE
            // failure-path test build only: the first stage of CTA 0 expects 16
            // bytes that no copy delivers, so the waits for it run out (the
            // copies it does issue all land before the CTA exits)
            if (blockIdx.x == 0 && blockIdx.y == 0 && stages == 0 && c0 == 0) bytes += 16;
#endif
            if (c0 + 32 >= n_here && lane == 0) mbar_arrive_expect_tx(smem_u32(&full[slot]), bytes);
            if (ok)
              bulk_g2s(sm0 + slot * stage_bytes + (c0 + lane) * page_bytes,
                       P.bounds + ((size_t)page * P.h_kv + g0) * 2 * D, copy_bytes,
                       smem_u32(&full[slot]));
          }
          ++stages;
          advance();
        }
      }
    } else {
      // ---------------------------------------------------------- scores
      const int gi = w % hs, sub = w / hs, g = g0 + gi;
      const bool works = sub < per_head && gi < heads;
      while (works && !stop && open()) {
        // lane i < 16: page i of this warp's 16 of a step, -1 where there is none
        auto page_at = [&](int k) {
          const int i = seg.p0 + k * stage_pages + sub * 16 + lane;
          if (lane >= 16 || i >= seg.p1) return -1;
          const int page = __ldg(seg.table + i);
          return page >= 0 && page < P.num_pages ? page : -1;
        };
        int page_cur = page_at(0), page_nxt = page_at(1);
        float sc = page_cur >= 0 ? __ldg(P.scales + (size_t)page_cur * P.h_kv + g) : 0.f;
        if (!waited) asm volatile("griddepcontrol.wait;\n" ::: "memory");  // the query's codes
        waited = true;
        // B fragments of the head's query codes: the column is a query head of
        // the group; the first D/32 k steps take the codes >= 0 (they meet the
        // max codes), the others those below 0
        uint32_t qb[NT][2 * KS][2];
        float t_q[NT][2];  // the scales of columns 2t and 2t + 1
        const size_t q0 = (size_t)seg.b * P.h_q + (size_t)g * P.group;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const int r = 8 * nt + (lane >> 2);
#pragma unroll
          for (int ks = 0; ks < KS; ++ks)
#pragma unroll
            for (int h = 0; h < 2; ++h)
              qb[nt][ks][h] = r < P.group ? __ldcg(reinterpret_cast<const uint32_t*>(
                                                P.q_codes + (q0 + r) * D + 32 * ks + 16 * h +
                                                4 * (lane & 3)))
                                          : 0u;
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int rq = 8 * nt + 2 * (lane & 3) + e;
            t_q[nt][e] = rq < P.group ? __ldcg(P.q_scales + q0 + rq) : 0.f;
          }
#pragma unroll
          for (int ks = 0; ks < KS; ++ks)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const uint32_t a = qb[nt][ks][h], neg = __vcmplts4(a, 0u);
              qb[nt][ks][h] = a & ~neg;
              qb[nt][KS + ks][h] = a & neg;
            }
        }
        float* out = P.scores + ((size_t)seg.b * P.h_kv + g) * P.row_stride;
        for (int k = 0; k < seg.steps; ++k) {
          // a step ahead: the next pages' scales, and the table entries behind them
          const float sc_nxt =
              page_nxt >= 0 ? __ldg(P.scales + (size_t)page_nxt * P.h_kv + g) : 0.f;
          const int page_nn = page_at(k + 2);
          if (!mbar_wait(smem_u32(&full[slot]), parity, &abort_flag)) {
            stop = true;
            break;
          }
          // 16 pages are the MMA's rows; every fragment is loaded, and the
          // stage given back, before the first is used
          const uint32_t rows = sm0 + slot * stage_bytes + (sub * 16 + (lane & 15)) * page_bytes +
                                gi * 2 * D + (lane >> 4) * 16;
          uint32_t x[2 * KS][4];
#pragma unroll
          for (int ks = 0; ks < 2 * KS; ++ks)
            ldmatrix_x4(rows + ks * 32, x[ks][0], x[ks][1], x[ks][2], x[ks][3]);
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&empty[slot]));
          advance();
          int acc[NT][2][4];  // two chains
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[nt][0][e] = acc[nt][1][e] = 0;
#pragma unroll
          for (int ks = 0; ks < 2 * KS; ++ks)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) mma_s8_16832(acc[nt][ks & 1], x[ks], qb[nt][ks]);
          // lane (g, t): pages g and g + 8, heads 2t and 2t + 1
          const float s0 = __shfl_sync(0xffffffffu, sc, lane >> 2);
          const float s1 = __shfl_sync(0xffffffffu, sc, (lane >> 2) + 8);
          float b0 = -INFINITY, b1 = -INFINITY;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              if (8 * nt + 2 * (lane & 3) + e < P.group) {
                // whole numbers below 2^24: exact as floats
                const float d0 = (float)(acc[nt][0][e] + acc[nt][1][e]);
                const float d1 = (float)(acc[nt][0][2 + e] + acc[nt][1][2 + e]);
                b0 = fmaxf(b0, __fmul_rn(__fmul_rn(d0, s0), t_q[nt][e]));
                b1 = fmaxf(b1, __fmul_rn(__fmul_rn(d1, s1), t_q[nt][e]));
              }
            }
#pragma unroll
          for (int o = 1; o < 4; o <<= 1) {
            b0 = fmaxf(b0, __shfl_xor_sync(0xffffffffu, b0, o));
            b1 = fmaxf(b1, __shfl_xor_sync(0xffffffffu, b1, o));
          }
          const int row = (lane >> 2) + 8 * (lane & 1);
          const int i = seg.p0 + k * stage_pages + sub * 16 + row;
          const int page = __shfl_sync(0xffffffffu, page_cur, row);
          if ((lane & 3) < 2 && i < seg.p1) out[i] = page >= 0 ? (lane & 1 ? b1 : b0) : -INFINITY;
          page_cur = page_nxt;
          page_nxt = page_nn;
          sc = sc_nxt;
        }
      }
    }
  }
  // no CTA ends before the query's kernel has, whether it read its codes or not
  asm volatile("griddepcontrol.wait;\n" ::: "memory");
  __syncthreads();  // every wait above is bounded
  // a wait that gave up: the copies in flight land before the CTA leaves (each
  // is the latest phase of its barrier)
  if (abort_flag && w == kScoreWarps)
    for (uint32_t i = stages > NST ? stages - NST : 0; i < stages; ++i)
      (void)mbar_drain(smem_u32(&full[i % NST]), (i / NST) & 1);
  if (tid == 0 && abort_flag) report(P.error_word, TL_DEVERR_TIMEOUT);
}

// ------------------------------------------------------------------ select --

struct PageSelectParams {
  const float* scores;
  int64_t row_stride;
  const int32_t* block_table;
  const int32_t* context_lens;
  int32_t* table;  // [B][h_kv][n]
  int32_t* lens;   // [B]
  int32_t max_pages_per_seq, h_kv, page_size, n, first, last;
  uint32_t* error_word;
};

template <int T, bool FITS>
__global__ void __launch_bounds__(T) page_select_kernel(PageSelectParams P, int csize, int key_cap) {
  __shared__ SelectShared<T> sh;
  extern __shared__ __align__(16) uint32_t sel_keys[];
  asm volatile("griddepcontrol.wait;\n" ::: "memory");
  const int row = (int)blockIdx.x >> (31 - __clz(csize)), rank = (int)blockIdx.x & (csize - 1);
  const int b = row / P.h_kv;
  const int L = P.context_lens[b];
  const int nb = blocks_of(L, P.max_pages_per_seq, P.page_size);
  if (row % P.h_kv == 0 && rank == 0 && threadIdx.x == 0) {
    P.lens[b] = nb == 0 ? 0 : nb <= P.n ? L : (P.n - 1) * P.page_size + (L - 1) % P.page_size + 1;
    if (nb == 0 && L > 0) report(P.error_word, TL_DEVERR_CONTEXT_RANGE);
  }
  const float* x = P.scores + (size_t)row * P.row_stride;
  const int32_t* from = P.block_table + (size_t)b * P.max_pages_per_seq;
  int32_t* to = P.table + (size_t)row * P.n;
  if (nb <= P.n) {  // every block
    for (int i = rank * T + threadIdx.x; i < P.n; i += csize * T)
      to[i] = i < nb ? __ldg(from + i) : -1;
    return;
  }
  const int2 mine = select_row<T, FITS>(
      sh, sel_keys, key_cap, x, nb, P.n, P.first, P.last, rank, csize,
      [&](int pos, int i) { to[pos] = i; }, [](int) {});
  __syncthreads();  // the CTA's blocks are in place: their table entries
  for (int pos = mine.x + threadIdx.x; pos < mine.y; pos += T) to[pos] = __ldg(from + to[pos]);
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
  // (block, head) pairs are counted in 32 bits
  if ((int64_t)B * max_pages_per_seq > INT32_MAX ||
      (int64_t)B * max_pages_per_seq * h_kv > INT32_MAX)
    return TL_ERR_UNSUPPORTED;
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
  const unsigned grid = (unsigned)std::min<int64_t>(most, (int64_t)num_sms() * bounds_ctas(kind));  // one wave
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
static bool launch_scores(const ScoreParams& P, cudaStream_t st) {
  const int64_t rows = (int64_t)P.B * P.h_q;
  page_query_kernel<D, QF32><<<(unsigned)((rows + 7) / 8), 256, 0, st>>>(P);
  if (launch_status() != TL_OK) return false;
  auto kernel = P.group <= 8 ? page_score_kernel<D, 1> : page_score_kernel<D, 2>;
  const int hs = score_heads(P.h_kv);
  // two CTAs share an SM's 228 KiB: at most (one head) 3 x 34 KiB of stages
  // each, 5 KiB of static state and the system's 1 KiB.  The limit is the same
  // whatever the heads: threads that launch different ones at once set it
  const int smem = kScoreStages * score_stage_bytes(hs, D);
  const int most = kScoreStages * score_stage_bytes(1, D);
  if (smem > most ||
      cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, most) != cudaSuccess)
    return false;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)num_sms() * 2, (unsigned)((P.h_kv + hs - 1) / hs));
  cfg.blockDim = dim3(kScoreThreads);
  cfg.dynamicSmemBytes = (size_t)smem;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, P) == cudaSuccess;
}

SelectShape select_shape(int64_t rows, int64_t cap) {
  SelectShape s;
  s.cluster = 1;
  // as many CTAs a row as its keys' shared memory asks for: a cluster's
  // barriers and remote reads cost more than the sweeps that it would divide
  // (8 rows of 128K values: 23.9 us by 4 CTAs each, 24.7 by 8)
  while (s.cluster < kSelClusterMax && cap > (int64_t)kSelKeysMax * s.cluster) s.cluster *= 2;
  const int64_t slice = ((cap + s.cluster - 1) / s.cluster + 127) / 128 * 128;
  s.keys = (int)std::min<int64_t>(slice, kSelKeysMax);
  s.fits = slice <= kSelKeysMax;  // else 1,024 threads, by the rule below
  const bool many = rows * s.cluster > 2 * num_sms();
  s.threads = slice <= 1024 || (many && slice <= 2048) ? 256 : many && slice <= 8192 ? 512 : 1024;
  return s;
}

cudaError_t launch_rows(const void* const (&kernels)[4], int64_t rows, const SelectShape& s,
                        void** args, bool dependent, cudaStream_t st) {
  const void* kernel = kernels[!s.fits ? 3 : s.threads == 256 ? 0 : s.threads == 512 ? 1 : 2];
  const int smem = s.keys * (int)sizeof(uint32_t);
  // the same limit for every shape: threads that launch different ones at once set it
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       kSelKeysMax * (int)sizeof(uint32_t));
  if (e != cudaSuccess) return e;
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
  cfg.dynamicSmemBytes = (size_t)smem;
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

namespace tl {
// Workspace of a selection: the scores, the query's scales and its codes.
struct SelectWorkspace {
  size_t q_scales, q_codes, bytes;
};
static SelectWorkspace select_ws_layout(int B, int h_q, int h_kv, int d, int max_pages) {
  SelectWorkspace w;
  w.q_scales = align_up(sizeof(float) * (size_t)B * h_kv * score_stride(max_pages), 256);
  w.q_codes = align_up(w.q_scales + sizeof(float) * (size_t)B * h_q, 256);
  w.bytes = align_up(w.q_codes + (size_t)B * h_q * d, 256);
  return w;
}
}  // namespace tl

extern "C" size_t tl_kv_page_select_workspace_size(int32_t B, int32_t h_q, int32_t h_kv, int32_t d,
                                                   int32_t max_pages_per_seq) {
  if (B <= 0 || h_q <= 0 || h_kv <= 0 || d <= 0 || max_pages_per_seq <= 0 || h_q % h_kv) return 0;
  return tl::select_ws_layout(B, h_q, h_kv, d, max_pages_per_seq).bytes;
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
  if ((d != 64 && d != 128) || h_q / h_kv > 16 || page_size > 256 ||
      (int64_t)B * max_pages_per_seq > INT32_MAX ||
      (int64_t)num_pages * page_size >= ((int64_t)1 << 31) ||
      (int64_t)n_select * page_size >= ((int64_t)1 << 31) ||
      (int64_t)B * h_kv > INT32_MAX / 8 || (h_kv + kScoreWarps - 1) / kScoreWarps > 65535)
    return TL_ERR_UNSUPPORTED;
  // places and blocks are counted in 32 bits, a step of all threads past the last one
  if (n_select > (1 << 30) || max_pages_per_seq > (1 << 30)) return TL_ERR_UNSUPPORTED;
  if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u) ||
      workspace_bytes < tl_kv_page_select_workspace_size(B, h_q, h_kv, d, max_pages_per_seq))
    return TL_ERR_WORKSPACE;
  // the selection's CTAs read lengths, tables and scores while others write: in
  // place, a head could see the length that another one's CTA has already cut
  const struct {
    const void* p;
    size_t bytes;
  } outs[] = {{page_table, sizeof(int32_t) * (size_t)B * h_kv * n_select},
              {page_lens, sizeof(int32_t) * (size_t)B}},
    read[] = {{context_lens, sizeof(int32_t) * (size_t)B},
              {block_table, sizeof(int32_t) * (size_t)B * max_pages_per_seq},
              {workspace, tl_kv_page_select_workspace_size(B, h_q, h_kv, d, max_pages_per_seq)}};
  for (const auto& o : outs)
    for (const auto& r : read)
      if (overlap(o.p, o.bytes, r.p, r.bytes)) return TL_ERR_INVALID_ARG;
  if (overlap(page_table, outs[0].bytes, page_lens, outs[1].bytes)) return TL_ERR_INVALID_ARG;
  cudaStream_t st = (cudaStream_t)stream;
  ScoreParams S;
  S.q = q;
  S.bounds = bounds;
  S.scales = bound_scales;
  S.block_table = block_table;
  S.context_lens = context_lens;
  const SelectWorkspace ws = select_ws_layout(B, h_q, h_kv, d, max_pages_per_seq);
  S.scores = static_cast<float*>(workspace);
  S.q_scales = reinterpret_cast<float*>(static_cast<char*>(workspace) + ws.q_scales);
  S.q_codes = reinterpret_cast<int8_t*>(static_cast<char*>(workspace) + ws.q_codes);
  S.row_stride = score_stride(max_pages_per_seq);
  S.max_pages_per_seq = max_pages_per_seq;
  S.B = B;
  S.h_q = h_q;
  S.h_kv = h_kv;
  S.group = h_q / h_kv;
  S.num_pages = num_pages;
  S.page_size = page_size;
  S.error_word = error_word;
  const bool f32 = q_dtype == TL_F32;
  const bool ran = d == 128 ? (f32 ? launch_scores<128, true>(S, st) : launch_scores<128, false>(S, st))
                            : (f32 ? launch_scores<64, true>(S, st) : launch_scores<64, false>(S, st));
  if (!ran) return TL_ERR_CUDA;
  PageSelectParams P;
  P.scores = S.scores;
  P.row_stride = S.row_stride;
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
  int csize = s.cluster, key_cap = s.keys;
  void* args[] = {&P, &csize, &key_cap};
  const void* const kernels[4] = {reinterpret_cast<const void*>(page_select_kernel<256, true>),
                                  reinterpret_cast<const void*>(page_select_kernel<512, true>),
                                  reinterpret_cast<const void*>(page_select_kernel<1024, true>),
                                  reinterpret_cast<const void*>(page_select_kernel<1024, false>)};
  if (launch_rows(kernels, rows, s, args, true, st) != cudaSuccess) return TL_ERR_CUDA;
  return launch_status();
}
