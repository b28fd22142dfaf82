// The decode entry points of the C ABI; the kernels and their launch are in
// paged_decode.cuh.
#include "paged_decode.cuh"

// ------------------------------------------------------------------- host --

extern "C" tl_status tl_decode_trace_reset(void) {
#if TL_DECODE_TRACE
  unsigned long long init[TL_TRACE_SLOTS] = {};
  init[TL_TRACE_COMBINE_START] = ~0ull;
  if (cudaDeviceSynchronize() != cudaSuccess) return TL_ERR_CUDA;
  if (cudaMemcpyToSymbol(tl::g_trace, init, sizeof(init)) != cudaSuccess) return TL_ERR_CUDA;
  return TL_OK;
#else
  return TL_ERR_UNSUPPORTED;
#endif
}

extern "C" tl_status tl_decode_trace_read(uint64_t* stamps, int32_t n) {
#if TL_DECODE_TRACE
  if (!stamps || n < 1 || n > TL_TRACE_SLOTS) return TL_ERR_INVALID_ARG;
  if (cudaDeviceSynchronize() != cudaSuccess) return TL_ERR_CUDA;
  if (cudaMemcpyFromSymbol(stamps, tl::g_trace, sizeof(uint64_t) * n) != cudaSuccess)
    return TL_ERR_CUDA;
  return TL_OK;
#else
  (void)stamps;
  (void)n;
  return TL_ERR_UNSUPPORTED;
#endif
}

extern "C" size_t tl_paged_attn_decode_workspace_size(int32_t B, int32_t h_q, int32_t h_kv,
                                                      int32_t d) {
  if (B <= 0 || h_q <= 0 || h_kv <= 0 || d <= 0 || h_q % h_kv) return 0;
  return tl::decode_ws_layout(B, h_q, h_kv, d, nullptr, nullptr);
}


extern "C" tl_status tl_paged_attn_decode(const void* q, const void* k_cache,
                                          const void* v_cache, const int32_t* block_table,
                                          int32_t max_pages_per_seq,
                                          const int32_t* context_lens, float* out, int32_t B,
                                          int32_t h_q, int32_t h_kv, int32_t d,
                                          int32_t num_pages, int32_t page_size, int32_t window,
                                          float scale, tl_dtype dtype, void* workspace,
                                          size_t workspace_bytes, uint32_t* error_word,
                                          void* stream) {
  return tl::decode_impl<false>(q, k_cache, v_cache, block_table, max_pages_per_seq, context_lens, out,
                         B, 1, h_q, h_kv, d, num_pages, page_size, window, 0, scale, dtype,
                         workspace, workspace_bytes, error_word, stream);
}

extern "C" tl_status tl_paged_attn_decode_int8(
    const void* q, const int8_t* k_codes, const int8_t* v_codes, const float* k_scales,
    const float* v_scales, const int32_t* block_table, int32_t max_pages_per_seq,
    const int32_t* context_lens, float* out, int32_t B, int32_t h_q, int32_t h_kv, int32_t d,
    int32_t num_pages, int32_t page_size, int32_t window, float scale, void* workspace,
    size_t workspace_bytes, uint32_t* error_word, void* stream) {
  if (!k_scales || !v_scales) return TL_ERR_INVALID_ARG;
  return tl::decode_impl<false>(q, k_codes, v_codes, block_table, max_pages_per_seq, context_lens, out,
                         B, 1, h_q, h_kv, d, num_pages, page_size, window, 0, scale,
                         TL_FP8_E4M3, workspace, workspace_bytes, error_word, stream,
                         tl::NewRows(), k_scales, v_scales);
}

extern "C" tl_status tl_paged_attn_decode_write_int8(
    const void* q, const void* k_new, const void* v_new, tl_dtype new_dtype,
    const int64_t* slot_mapping, int32_t n_new, int8_t* k_codes, int8_t* v_codes,
    float* k_scales, float* v_scales, const int32_t* block_table, int32_t max_pages_per_seq,
    const int32_t* context_lens, float* out, int32_t B, int32_t h_q, int32_t h_kv, int32_t d,
    int32_t num_pages, int32_t page_size, int32_t window, float scale, void* workspace,
    size_t workspace_bytes, uint32_t* error_word, void* stream) {
  if (!k_scales || !v_scales) return TL_ERR_INVALID_ARG;
  tl::NewRows nr;
  nr.k_new = k_new;
  nr.v_new = v_new;
  nr.slot_mapping = slot_mapping;
  nr.n = n_new;
  nr.new_dtype = new_dtype;
  nr.k_dst = k_codes;
  nr.v_dst = v_codes;
  return tl::decode_impl<false>(q, k_codes, v_codes, block_table, max_pages_per_seq, context_lens, out,
                         B, 1, h_q, h_kv, d, num_pages, page_size, window, 0, scale,
                         TL_FP8_E4M3, workspace, workspace_bytes, error_word, stream, nr,
                         k_scales, v_scales);
}

extern "C" tl_status tl_paged_attn_decode_write(
    const void* q, const void* k_new, const void* v_new, tl_dtype new_dtype,
    const int64_t* slot_mapping, int32_t n_new, void* k_cache, void* v_cache,
    const int32_t* block_table, int32_t max_pages_per_seq, const int32_t* context_lens,
    float* out, int32_t B, int32_t h_q, int32_t h_kv, int32_t d, int32_t num_pages,
    int32_t page_size, int32_t window, float scale, tl_dtype dtype, void* workspace,
    size_t workspace_bytes, uint32_t* error_word, void* stream) {
  tl::NewRows nr;
  nr.k_new = k_new;
  nr.v_new = v_new;
  nr.slot_mapping = slot_mapping;
  nr.n = n_new;
  nr.new_dtype = new_dtype;
  nr.k_dst = k_cache;
  nr.v_dst = v_cache;
  return tl::decode_impl<false>(q, k_cache, v_cache, block_table, max_pages_per_seq, context_lens, out,
                         B, 1, h_q, h_kv, d, num_pages, page_size, window, 0, scale, dtype,
                         workspace, workspace_bytes, error_word, stream, nr);
}

extern "C" tl_status tl_paged_attn_decode_write_ring(
    const void* q, const void* k_new, const void* v_new, tl_dtype new_dtype,
    const int64_t* slot_mapping, int32_t n_new, void* k_cache, void* v_cache,
    const int32_t* block_table, int32_t max_pages_per_seq, const int32_t* context_lens,
    float* out, int32_t B, int32_t h_q, int32_t h_kv, int32_t d, int32_t num_pages,
    int32_t page_size, int32_t window, int32_t ring_pages, float scale, tl_dtype dtype,
    void* workspace, size_t workspace_bytes, uint32_t* error_word, void* stream) {
  if (ring_pages <= 0 || ring_pages > max_pages_per_seq || window <= 0 || page_size <= 0 ||
      (int64_t)ring_pages * page_size < window)
    return TL_ERR_INVALID_ARG;
  tl::NewRows nr;
  nr.k_new = k_new;
  nr.v_new = v_new;
  nr.slot_mapping = slot_mapping;
  nr.n = n_new;
  nr.new_dtype = new_dtype;
  nr.k_dst = k_cache;
  nr.v_dst = v_cache;
  return tl::decode_impl<false>(q, k_cache, v_cache, block_table, max_pages_per_seq, context_lens, out,
                         B, 1, h_q, h_kv, d, num_pages, page_size, window, ring_pages, scale,
                         dtype, workspace, workspace_bytes, error_word, stream, nr);
}

extern "C" tl_status tl_paged_attn_decode_ring(
    const void* q, const void* k_cache, const void* v_cache, const int32_t* block_table,
    int32_t max_pages_per_seq, const int32_t* context_lens, float* out, int32_t B, int32_t h_q,
    int32_t h_kv, int32_t d, int32_t num_pages, int32_t page_size, int32_t window,
    int32_t ring_pages, float scale, tl_dtype dtype, void* workspace, size_t workspace_bytes,
    uint32_t* error_word, void* stream) {
  // the ring must be part of the table and must hold one window
  if (ring_pages <= 0 || ring_pages > max_pages_per_seq || window <= 0 || page_size <= 0 ||
      (int64_t)ring_pages * page_size < window)
    return TL_ERR_INVALID_ARG;
  return tl::decode_impl<false>(q, k_cache, v_cache, block_table, max_pages_per_seq, context_lens, out,
                         B, 1, h_q, h_kv, d, num_pages, page_size, window, ring_pages, scale,
                         dtype, workspace, workspace_bytes, error_word, stream);
}

extern "C" tl_status tl_paged_attn_decode_ring_int8(
    const void* q, const int8_t* k_codes, const int8_t* v_codes, const float* k_scales,
    const float* v_scales, const int32_t* block_table, int32_t max_pages_per_seq,
    const int32_t* context_lens, float* out, int32_t B, int32_t h_q, int32_t h_kv, int32_t d,
    int32_t num_pages, int32_t page_size, int32_t window, int32_t ring_pages, float scale,
    void* workspace, size_t workspace_bytes, uint32_t* error_word, void* stream) {
  if (!k_scales || !v_scales) return TL_ERR_INVALID_ARG;
  // the ring must be part of the table and must hold one window
  if (ring_pages <= 0 || ring_pages > max_pages_per_seq || window <= 0 || page_size <= 0 ||
      (int64_t)ring_pages * page_size < window)
    return TL_ERR_INVALID_ARG;
  return tl::decode_impl<false>(q, k_codes, v_codes, block_table, max_pages_per_seq, context_lens, out,
                         B, 1, h_q, h_kv, d, num_pages, page_size, window, ring_pages, scale,
                         TL_FP8_E4M3, workspace, workspace_bytes, error_word, stream,
                         tl::NewRows(), k_scales, v_scales);
}

extern "C" size_t tl_paged_attn_decode_multi_workspace_size(int32_t B, int32_t q_len,
                                                            int32_t h_q, int32_t h_kv, int32_t d) {
  if (B <= 0 || q_len <= 0 || h_q <= 0 || h_kv <= 0 || d <= 0 || h_q % h_kv) return 0;
  return tl::decode_ws_layout(B, q_len * h_q, h_kv, d, nullptr, nullptr);
}

extern "C" tl_status tl_paged_attn_decode_multi_int8(
    const void* q, const int8_t* k_codes, const int8_t* v_codes, const float* k_scales,
    const float* v_scales, const int32_t* block_table, int32_t max_pages_per_seq,
    const int32_t* context_lens, float* out, int32_t B, int32_t q_len, int32_t h_q, int32_t h_kv,
    int32_t d, int32_t num_pages, int32_t page_size, int32_t window, float scale,
    void* workspace, size_t workspace_bytes, uint32_t* error_word, void* stream) {
  if (!k_scales || !v_scales) return TL_ERR_INVALID_ARG;
  return tl::decode_impl<false>(q, k_codes, v_codes, block_table, max_pages_per_seq, context_lens, out,
                         B, q_len, h_q, h_kv, d, num_pages, page_size, window, 0, scale,
                         TL_FP8_E4M3, workspace, workspace_bytes, error_word, stream,
                         tl::NewRows(), k_scales, v_scales);
}

extern "C" tl_status tl_paged_attn_decode_multi(
    const void* q, const void* k_cache, const void* v_cache, const int32_t* block_table,
    int32_t max_pages_per_seq, const int32_t* context_lens, float* out, int32_t B, int32_t q_len,
    int32_t h_q, int32_t h_kv, int32_t d, int32_t num_pages, int32_t page_size, int32_t window,
    float scale, tl_dtype dtype, void* workspace, size_t workspace_bytes, uint32_t* error_word,
    void* stream) {
  return tl::decode_impl<false>(q, k_cache, v_cache, block_table, max_pages_per_seq, context_lens, out,
                         B, q_len, h_q, h_kv, d, num_pages, page_size, window, 0, scale, dtype,
                         workspace, workspace_bytes, error_word, stream);
}
