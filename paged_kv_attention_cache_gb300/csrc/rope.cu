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

static tl_status launch_rope(const RopeRows& R, bool f32, int kind, cudaStream_t st) {
  const int heads = R.h_q + (R.slots ? 2 * R.h_kv : 0);
  const int64_t rows = (int64_t)R.n * heads;
  const unsigned blocks =
      (unsigned)std::min<int64_t>((rows + 7) / 8, (int64_t)num_sms() * 64);
  auto kern = f32 ? (kind == kRopeSame   ? rope_rows_kernel<true, kRopeSame>
                     : kind == kRopeE4m3 ? rope_rows_kernel<true, kRopeE4m3>
                                         : rope_rows_kernel<true, kRopeInt8>)
                  : (kind == kRopeSame   ? rope_rows_kernel<false, kRopeSame>
                     : kind == kRopeE4m3 ? rope_rows_kernel<false, kRopeE4m3>
                                         : rope_rows_kernel<false, kRopeInt8>);
  kern<<<blocks, 256, 0, st>>>(R, heads);
  return launch_status();
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
  *rope_scale = scaling == TL_ROPE_RAMP ? (float)(0.1 * std::log(factor) + 1.0) : 1.f;
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
