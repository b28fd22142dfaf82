// Host-side checks of the calls that rotate rows (rope.cu and the decode call
// that rotates and writes its new rows itself).
#pragma once

#include "rope.cuh"

namespace tl {

constexpr int kRopeMaxDim = 4096;  // elements of a row

// Whether rows of na elements at a + t * sa and nb at b + t * sb, t < n, have
// an element in common (strides in elements of `elem` bytes).  Rows of one
// stride, as parts of one tensor's rows, are told apart exactly; of different
// strides by the ranges they span.
inline bool rows_overlap(const void* a, int64_t sa, int64_t na, const void* b, int64_t sb,
                         int64_t nb, int64_t n, int elem) {
  if (!overlap(a, (size_t)((n - 1) * sa + na) * elem, b, (size_t)((n - 1) * sb + nb) * elem))
    return false;
  if (n == 1 || sa != sb || sa < na || sa < nb) return true;
  const intptr_t step = (intptr_t)sa * elem;
  intptr_t by = (intptr_t)(reinterpret_cast<uintptr_t>(b) - reinterpret_cast<uintptr_t>(a)) % step;
  if (by < 0) by += step;
  return by < (intptr_t)na * elem || by + (intptr_t)nb * elem > step;
}

inline bool aligned_to(const void* p, int bytes) {
  return (reinterpret_cast<uintptr_t>(p) & (uintptr_t)(bytes - 1)) == 0;
}

// The width W of the rotary units' words in which a call's rows can be moved: 16
// bytes' elements, or 2; 0: neither (element by element).
inline int rope_unit_width(const RopeRows& R, int elem) {
  if (R.d % 16 || R.d > 16 * kRopeMaxUnits) return 0;
  for (const int W : {16 / elem, 2}) {
    auto row = [&](const void* p, int64_t stride) {
      return aligned_to(p, W * elem) && stride % W == 0;
    };
    if (R.rot % (R.interleaved ? W : 2 * W) == 0 && row(R.q, R.q_stride) &&
        row(R.q_out, R.out_stride) && row(R.k, R.k_stride) && row(R.v, R.v_stride))
      return W;
  }
  return 0;
}

// n > 0 rows of `row` elements read at x and written at out.
inline tl_status rope_io_checked(const void* x, int64_t x_stride, const void* out,
                                 int64_t out_stride, int64_t n, int64_t row, int elem) {
  if (!x || !out || !aligned_to(x, elem) || !aligned_to(out, elem)) return TL_ERR_INVALID_ARG;
  if (n == 1) x_stride = out_stride = row;
  if (x_stride < 0 || out_stride < row || x_stride > ((int64_t)1 << 30) ||
      out_stride > ((int64_t)1 << 30))
    return TL_ERR_INVALID_ARG;
  const bool in_place = x == out && x_stride == out_stride;
  if (!in_place && rows_overlap(x, x_stride, row, out, out_stride, row, n, elem))
    return TL_ERR_INVALID_ARG;
  return TL_OK;
}

// Whether what a call of n tokens writes (bytes at p) has a byte in common with
// the lists that its other warps read: positions, the frequencies, and slots
// (null: none).
inline bool over_rope_lists(const void* p, size_t bytes, const int64_t* slots,
                            const int32_t* positions, const uint64_t* freqs, int32_t n,
                            int32_t rot_dim) {
  return overlap(p, bytes, positions, sizeof(int32_t) * (size_t)n) ||
         overlap(p, bytes, freqs, sizeof(uint64_t) * (size_t)(rot_dim / 2)) ||
         (slots && overlap(p, bytes, slots, sizeof(int64_t) * (size_t)n));
}

// The checks of an append's arguments (sizes positive, n_tokens >= 0); with
// tokens, *R and the rows' kind.  dtype TL_INT8: codes and scales.
inline tl_status rope_rows_checked(const void* q, int64_t q_stride, void* q_out,
                                   int64_t q_out_stride, const void* k_new, int64_t k_stride,
                                   const void* v_new, int64_t v_stride, tl_dtype src_dtype,
                                   void* k_dst, void* v_dst, float* k_scales, float* v_scales,
                                   const int64_t* slots, const int32_t* positions,
                                   const uint64_t* freqs, int32_t rot_dim, int32_t interleaved,
                                   float rope_scale, int32_t n, int32_t num_pages,
                                   int32_t page_size, int32_t h_q, int32_t h_kv, int32_t d,
                                   tl_dtype dtype, uint32_t* error_word, RopeRows* R, int* kind) {
  if (rot_dim < 2 || rot_dim % 2 || rot_dim > d) return TL_ERR_INVALID_ARG;
  if (src_dtype != TL_F32 && src_dtype != TL_BF16) return TL_ERR_UNSUPPORTED;
  if (dtype != src_dtype && dtype != TL_FP8_E4M3 && dtype != TL_INT8) return TL_ERR_UNSUPPORTED;
  if (d > (dtype == TL_INT8 ? 1024 : kRopeMaxDim) ||
      ((int64_t)h_q + 2 * (int64_t)h_kv) * d > INT32_MAX ||
      (int64_t)num_pages * page_size > INT32_MAX)
    return TL_ERR_UNSUPPORTED;
  if (n == 0) return TL_OK;
  if (!k_new || !v_new || !k_dst || !v_dst || !slots || !positions || !freqs ||
      (h_q > 0) != (q != nullptr) || (h_q > 0) != (q_out != nullptr) ||
      (dtype == TL_INT8 && (!k_scales || !v_scales)))
    return TL_ERR_INVALID_ARG;
  const int elem = src_dtype == TL_F32 ? 4 : 2;
  const int pool_elem = dtype == TL_F32 ? 4 : dtype == TL_BF16 ? 2 : 1;
  const int64_t row = (int64_t)h_kv * d, q_row = (int64_t)h_q * d;
  if (!aligned_to(k_new, elem) || !aligned_to(v_new, elem) || !aligned16(k_dst) ||
      !aligned16(v_dst) || !aligned_to(k_scales, 4) || !aligned_to(v_scales, 4) ||
      !aligned_to(slots, 8) || !aligned_to(positions, 4) || !aligned_to(freqs, 8) ||
      row * pool_elem % 16)
    return TL_ERR_INVALID_ARG;
  if (n == 1) {
    k_stride = v_stride = row;
    q_stride = q_out_stride = q_row;
  }
  const int64_t most = (int64_t)1 << 30;
  if (k_stride < 0 || v_stride < 0 || k_stride > most || v_stride > most)
    return TL_ERR_INVALID_ARG;
  if (h_q > 0) {
    const tl_status ok = rope_io_checked(q, q_stride, q_out, q_out_stride, n, q_row, elem);
    if (ok != TL_OK) return ok;
    if (rows_overlap(q_out, q_out_stride, q_row, k_new, k_stride, row, n, elem) ||
        rows_overlap(q_out, q_out_stride, q_row, v_new, v_stride, row, n, elem))
      return TL_ERR_INVALID_ARG;
  }
  // what is written against everything else that is read or written
  const size_t slots_all = (size_t)num_pages * page_size;
  const size_t pool = slots_all * row * pool_elem;
  const size_t scales = dtype == TL_INT8 ? slots_all * h_kv * sizeof(float) : 0;
  const struct {
    const void* p;
    size_t bytes;
  } spans[] = {{k_dst, pool},
               {v_dst, pool},
               {k_scales, scales},
               {v_scales, scales},
               {k_new, (size_t)((n - 1) * k_stride + row) * elem},
               {v_new, (size_t)((n - 1) * v_stride + row) * elem},
               {q, h_q > 0 ? (size_t)((n - 1) * q_stride + q_row) * elem : 0},
               {q_out, h_q > 0 ? (size_t)((n - 1) * q_out_stride + q_row) * elem : 0}};
  for (int i = 0; i < 4; ++i)
    for (int j = i + 1; j < 8; ++j)
      if (spans[i].bytes && spans[j].bytes &&
          overlap(spans[i].p, spans[i].bytes, spans[j].p, spans[j].bytes))
        return TL_ERR_INVALID_ARG;
  for (int i : {0, 1, 2, 3, 7})
    if (spans[i].bytes &&
        over_rope_lists(spans[i].p, spans[i].bytes, slots, positions, freqs, n, rot_dim))
      return TL_ERR_INVALID_ARG;
  *R = RopeRows();
  R->q = q;
  R->k = k_new;
  R->v = v_new;
  R->q_out = q_out;
  R->q_stride = q_stride;
  R->k_stride = k_stride;
  R->v_stride = v_stride;
  R->out_stride = q_out_stride;
  R->k_dst = k_dst;
  R->v_dst = v_dst;
  R->k_scales = k_scales;
  R->v_scales = v_scales;
  R->slots = slots;
  R->positions = positions;
  R->freqs = freqs;
  R->n_slots = (int64_t)slots_all;
  R->n = n;
  R->h_q = h_q;
  R->h_kv = h_kv;
  R->d = d;
  R->rot = rot_dim;
  R->page_size = page_size;
  R->interleaved = interleaved != 0;
  R->scale = rope_scale;
  R->error_word = error_word;
  *kind = dtype == TL_INT8 ? kRopeInt8 : dtype == TL_FP8_E4M3 ? kRopeE4m3 : kRopeSame;
  return TL_OK;
}

}  // namespace tl
