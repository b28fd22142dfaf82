// Rotary positions: the tables (host), the rotation of query or key rows, and
// the append that rotates queries and keys on their way to q_out and the pages.
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "rope.cuh"
#include "rope_host.h"

namespace tl {

// One warp per (token, head).
template <bool F32, int KIND>
__global__ void __launch_bounds__(256) rope_rows_kernel(RopeRows R, int heads) {
  const int lane = threadIdx.x & 31;
  const int64_t stride = (int64_t)gridDim.x * (blockDim.x >> 5);
  const int64_t rows = (int64_t)R.n * heads;
  for (int64_t r = (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5); r < rows;
       r += stride)
    rope_row<F32, KIND>(R, r / heads, (int)(r % heads), lane);
}

// One warp per item: P passes over a token's heads.  Bound: HBM (each row read
// and written once).  What it took, on 16,384 tokens of 32 bf16 heads of 128
// (268 MB) and on a prompts' append of 12,288 such tokens with 8 KV heads (369
// MB, copies included):
//   one warp a (token, head), an element pair a lane  127 us   175 us
//   one pass of 4 heads a warp, 256 threads            59        89
//   two passes                                         46        63
//   four, streaming accesses, 80 registers             43        56
//   four, CTAs of two warps                            41.5      54.8 (6.7 TB/s)
// (f32, two passes: 78.4 and 107 us, 6.9 TB/s; e4m3 and int8 pools, two passes:
// 61 and 74 us for the append, instruction issue beside the bytes, the int8
// rows' quotients above all; rot 120 of 128, in words of two elements: 51 and
// 70 us, element by element 135 and 179.)
// Passes amortise a token's angles and keep more loads in flight; beyond the
// registers of three 256-thread CTAs an SM they spill (four f32 passes 34 us
// against 20 with two).  Small CTAs give their registers back as soon as their
// own rows are written (512 threads: 51 and 69 us).
constexpr int kRopeThreads = 64;
template <bool F32, int KIND, bool INTER, int P, int W>
__global__ void __launch_bounds__(kRopeThreads, 768 / kRopeThreads)
    rope_units_kernel(RopeRows R, int heads, int U, int HW, uint32_t per_token, uint32_t items) {
  constexpr int warps = kRopeThreads / 32;
  __shared__ float4 cs[warps][4 * kRopeMaxUnits];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint32_t i = blockIdx.x * warps + warp;
  if (i >= items) return;
  const uint32_t t = i / per_token;
  rope_units<F32, KIND, INTER, P, W>(R, t, (int)(i - t * per_token) * P * HW, heads, U, HW, lane,
                                  cs[warp]);
}

// The most passes: as many as keep a kernel in its 80 registers (W: see
// rope_unit_width; words of 2 elements take more addresses).
template <bool F32, int KIND, int W>
constexpr int kRopePasses = (KIND == kRopeSame && W > 2 ? 4 : 2) / (F32 ? 2 : 1);

template <bool F32, int KIND, int W>
static tl_status launch_units(const RopeRows& R, int heads, cudaStream_t st) {
  const int U = R.d / 16, HW = 32 / U, passes = (heads + HW - 1) / HW;
  // fewer where a token has fewer, and while warps are few: 64 tokens of a
  // decode step take 2.5 us with one pass, 2.7 with two and 3.4 with four
  int P = kRopePasses<F32, KIND, W>;
  while (P > 1 && (P > passes || (int64_t)R.n * ((passes + P - 1) / P) < 16 * (int64_t)num_sms()))
    P /= 2;
  const uint32_t per_token = (passes + P - 1) / P, items = R.n * per_token;
  const unsigned grid = (items + kRopeThreads / 32 - 1) / (kRopeThreads / 32);
  auto launch = [&](auto kern) {
    kern<<<grid, kRopeThreads, 0, st>>>(R, heads, U, HW, per_token, items);
    return launch_status();
  };
  if constexpr (kRopePasses<F32, KIND, W> >= 4)
    if (P == 4)
      return R.interleaved ? launch(rope_units_kernel<F32, KIND, true, 4, W>)
                           : launch(rope_units_kernel<F32, KIND, false, 4, W>);
  if constexpr (kRopePasses<F32, KIND, W> >= 2)
    if (P == 2)
      return R.interleaved ? launch(rope_units_kernel<F32, KIND, true, 2, W>)
                           : launch(rope_units_kernel<F32, KIND, false, 2, W>);
  return R.interleaved ? launch(rope_units_kernel<F32, KIND, true, 1, W>)
                       : launch(rope_units_kernel<F32, KIND, false, 1, W>);
}

template <bool F32, int KIND>
static tl_status launch_rows(const RopeRows& R, cudaStream_t st) {
  const int heads = R.h_q + (R.slots ? 2 * R.h_kv : 0);
  // (items of a pass are counted in 32 bits)
  if ((int64_t)R.n * heads < ((int64_t)1 << 31)) {
    const int W = rope_unit_width(R, F32 ? 4 : 2);
    if (W > 2) return launch_units<F32, KIND, F32 ? 4 : 8>(R, heads, st);
    if (W == 2) return launch_units<F32, KIND, 2>(R, heads, st);
  }
  // a warp a row, element by element
  const int64_t rows = (int64_t)R.n * heads;
  const unsigned blocks = (unsigned)std::min<int64_t>((rows + 7) / 8, (int64_t)num_sms() * 64);
  rope_rows_kernel<F32, KIND><<<blocks, 256, 0, st>>>(R, heads);
  return launch_status();
}

static tl_status launch_rope(const RopeRows& R, bool f32, int kind, cudaStream_t st) {
  if (f32)
    return kind == kRopeSame   ? launch_rows<true, kRopeSame>(R, st)
           : kind == kRopeE4m3 ? launch_rows<true, kRopeE4m3>(R, st)
                               : launch_rows<true, kRopeInt8>(R, st);
  return kind == kRopeSame   ? launch_rows<false, kRopeSame>(R, st)
         : kind == kRopeE4m3 ? launch_rows<false, kRopeE4m3>(R, st)
                             : launch_rows<false, kRopeInt8>(R, st);
}

static tl_status write_rope_impl(const void* q, int64_t q_stride, void* q_out,
                                 int64_t q_out_stride, const void* k_new, int64_t k_stride,
                                 const void* v_new, int64_t v_stride, tl_dtype src_dtype,
                                 void* k_dst, void* v_dst, float* k_scales, float* v_scales,
                                 const int64_t* slot_mapping, const int32_t* positions,
                                 const uint64_t* freqs, int32_t rot_dim, int32_t interleaved,
                                 float rope_scale, int32_t n_tokens, int32_t num_pages,
                                 int32_t page_size, int32_t h_q, int32_t h_kv, int32_t d,
                                 tl_dtype dtype, uint32_t* error_word, void* stream) {
  if (n_tokens < 0 || num_pages <= 0 || page_size <= 0 || h_q < 0 || h_kv <= 0 || d <= 0)
    return TL_ERR_INVALID_ARG;
  RopeRows R;
  int kind;
  const tl_status ok = rope_rows_checked(
      q, q_stride, q_out, q_out_stride, k_new, k_stride, v_new, v_stride, src_dtype, k_dst, v_dst,
      k_scales, v_scales, slot_mapping, positions, freqs, rot_dim, interleaved, rope_scale,
      n_tokens, num_pages, page_size, h_q, h_kv, d, dtype, error_word, &R, &kind);
  if (ok != TL_OK || n_tokens == 0) return ok;
  return launch_rope(R, src_dtype == TL_F32, kind, (cudaStream_t)stream);
}

}  // namespace tl

// -------------------------------------------------------------------- host --

extern "C" tl_status tl_rope_freqs(int32_t rot_dim, double base, int32_t scaling, double factor,
                                   double trained_len, double low, double high,
                                   const double* factors, uint64_t* freqs, float* rope_scale) {
  if (rot_dim < 2 || rot_dim > 4096 || rot_dim % 2 || !freqs || !rope_scale)
    return TL_ERR_INVALID_ARG;
  if (scaling < TL_ROPE_PLAIN || scaling > TL_ROPE_FACTORS) return TL_ERR_UNSUPPORTED;
  if (!(base > 1.0) || !std::isfinite(base)) return TL_ERR_INVALID_ARG;
  const bool uses_factor = scaling != TL_ROPE_PLAIN && scaling != TL_ROPE_FACTORS;
  const bool uses_turns = scaling == TL_ROPE_BANDS || scaling == TL_ROPE_RAMP;
  if (uses_factor && (!(factor > 0.0) || !std::isfinite(factor))) return TL_ERR_INVALID_ARG;
  if (uses_turns && (!(trained_len > 0.0) || !std::isfinite(trained_len) || !(low > 0.0) ||
                     !(high > low) || !std::isfinite(high)))
    return TL_ERR_INVALID_ARG;
  const int n = rot_dim / 2;
  if (scaling == TL_ROPE_FACTORS) {
    if (!factors) return TL_ERR_INVALID_ARG;
    for (int i = 0; i < n; ++i)
      if (!(factors[i] > 0.0) || !std::isfinite(factors[i])) return TL_ERR_INVALID_ARG;
  }
  const double pi = 3.14159265358979323846;
  if (scaling == TL_ROPE_BASE) {
    if (rot_dim <= 2) return TL_ERR_INVALID_ARG;
    base *= std::pow(factor, (double)rot_dim / (rot_dim - 2));
    if (!(base > 1.0) || !std::isfinite(base)) return TL_ERR_INVALID_ARG;
  }
  // the (fractional) index of the pair that makes `turns` turns over the trained length
  auto index_of = [&](double turns) {
    return rot_dim * std::log(trained_len / (turns * 2 * pi)) / (2 * std::log(base));
  };
  double from = 0, to = 0;
  if (scaling == TL_ROPE_RAMP) {
    from = std::max(std::floor(index_of(high)), 0.0);
    to = std::min(std::ceil(index_of(low)), rot_dim - 1.0);
  }
  for (int i = 0; i < n; ++i) {
    double f = std::pow(base, -2.0 * i / rot_dim);
    double slow = scaling == TL_ROPE_LINEAR ? 1.0 : 0.0;  // how much of f / factor
    if (scaling == TL_ROPE_BANDS)
      slow = 1 - std::min(std::max((trained_len * f / (2 * pi) - low) / (high - low), 0.0), 1.0);
    if (scaling == TL_ROPE_RAMP)
      slow = std::min(std::max((i - from) / std::max(to - from, 1e-3), 0.0), 1.0);
    if (slow > 0) f = f / factor * slow + f * (1 - slow);
    if (scaling == TL_ROPE_FACTORS) f /= factors[i];
    const double turns = f / (2 * pi);
    if (!std::isfinite(turns)) return TL_ERR_INVALID_ARG;
    // the fraction of a turn in [0, 1): 2^64 of them, nearest; a fraction that
    // rounds up to 1 is a whole turn, 0
    const double part = std::rint((turns - std::floor(turns)) * 0x1p64);
    freqs[i] = part >= 0x1p64 ? 0 : (uint64_t)part;
  }
  *rope_scale =
      scaling == TL_ROPE_RAMP && factor > 1.0 ? (float)(0.1 * std::log(factor) + 1.0) : 1.f;
  return TL_OK;
}

extern "C" tl_status tl_rope(const void* x, int64_t x_stride, void* out, int64_t out_stride,
                             const int32_t* positions, const uint64_t* freqs, int32_t rot_dim,
                             int32_t interleaved, float rope_scale, int32_t n_tokens,
                             int32_t heads, int32_t d, tl_dtype dtype, void* stream) {
  using namespace tl;
  if (n_tokens < 0 || heads <= 0 || d <= 0 || rot_dim < 2 || rot_dim % 2 || rot_dim > d)
    return TL_ERR_INVALID_ARG;
  if (dtype != TL_F32 && dtype != TL_BF16) return TL_ERR_UNSUPPORTED;
  if (d > kRopeMaxDim || (int64_t)heads * d > INT32_MAX) return TL_ERR_UNSUPPORTED;
  if (n_tokens == 0) return TL_OK;
  if (!positions || !freqs || (reinterpret_cast<uintptr_t>(positions) & 3u) ||
      (reinterpret_cast<uintptr_t>(freqs) & 7u))
    return TL_ERR_INVALID_ARG;
  const int elem = dtype == TL_F32 ? 4 : 2;
  const tl_status ok = rope_io_checked(x, x_stride, out, out_stride, n_tokens, heads * d, elem);
  if (ok != TL_OK) return ok;
  const int64_t row = (int64_t)heads * d;
  if (over_rope_lists(out, (size_t)((n_tokens > 1 ? n_tokens - 1 : 0) * out_stride + row) * elem,
                      nullptr, positions, freqs, n_tokens, rot_dim))
    return TL_ERR_INVALID_ARG;
  RopeRows R = {};
  R.q = x;
  R.q_out = out;
  R.q_stride = n_tokens > 1 ? x_stride : 0;
  R.out_stride = n_tokens > 1 ? out_stride : 0;
  R.positions = positions;
  R.freqs = freqs;
  R.n = n_tokens;
  R.h_q = heads;
  R.d = d;
  R.rot = rot_dim;
  R.interleaved = interleaved != 0;
  R.scale = rope_scale;
  return launch_rope(R, dtype == TL_F32, kRopeSame, (cudaStream_t)stream);
}

extern "C" tl_status tl_kv_cache_write_rope(
    const void* q, int64_t q_stride, void* q_out, int64_t q_out_stride, const void* k_new,
    int64_t k_stride, const void* v_new, int64_t v_stride, tl_dtype src_dtype, void* k_cache,
    void* v_cache, const int64_t* slot_mapping, const int32_t* positions, const uint64_t* freqs,
    int32_t rot_dim, int32_t interleaved, float rope_scale, int32_t n_tokens, int32_t num_pages,
    int32_t page_size, int32_t h_q, int32_t h_kv, int32_t d, tl_dtype dtype,
    uint32_t* error_word, void* stream) {
  return tl::write_rope_impl(q, q_stride, q_out, q_out_stride, k_new, k_stride, v_new, v_stride,
                             src_dtype, k_cache, v_cache, nullptr, nullptr, slot_mapping,
                             positions, freqs, rot_dim, interleaved, rope_scale, n_tokens,
                             num_pages, page_size, h_q, h_kv, d, dtype, error_word, stream);
}

extern "C" tl_status tl_kv_cache_write_rope_int8(
    const void* q, int64_t q_stride, void* q_out, int64_t q_out_stride, const void* k_new,
    int64_t k_stride, const void* v_new, int64_t v_stride, tl_dtype src_dtype, int8_t* k_codes,
    int8_t* v_codes, float* k_scales, float* v_scales, const int64_t* slot_mapping,
    const int32_t* positions, const uint64_t* freqs, int32_t rot_dim, int32_t interleaved,
    float rope_scale, int32_t n_tokens, int32_t num_pages, int32_t page_size, int32_t h_q,
    int32_t h_kv, int32_t d, uint32_t* error_word, void* stream) {
  return tl::write_rope_impl(q, q_stride, q_out, q_out_stride, k_new, k_stride, v_new, v_stride,
                             src_dtype, k_codes, v_codes, k_scales, v_scales, slot_mapping,
                             positions, freqs, rot_dim, interleaved, rope_scale, n_tokens,
                             num_pages, page_size, h_q, h_kv, d, TL_INT8, error_word, stream);
}
