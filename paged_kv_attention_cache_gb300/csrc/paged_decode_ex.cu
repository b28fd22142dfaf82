// Decode over a table of selected pages per (sequence, KV head), and decode
// that adds every key's softmax probability to a running mass: the EX form of
// the decode kernels (paged_decode.cuh).  The pages of this library's model
// ("How serving works in Tlaloc") name neither; both serve contexts too long
// to read whole at every step.
#include "paged_decode.cuh"

namespace tl {

// Workspace of a mass call: the decode's, the rows' statistics, the scores.
struct MassWorkspace {
  size_t stats, scores, bytes;
  int64_t score_stride;
};

static MassWorkspace mass_ws_layout(int B, int q_len, int h_q, int h_kv, int d, int mass_len) {
  MassWorkspace w;
  // a row of scores takes whole 16-key chunks, at 128-byte steps
  w.score_stride = (int64_t)align_up((size_t)mass_len, 32);
  w.stats = align_up(decode_ws_layout(B, q_len * h_q, h_kv, d, nullptr, nullptr), 256);
  w.scores = align_up(w.stats + sizeof(float) * 2 * (size_t)B * q_len * h_q, 256);
  w.bytes = w.scores + sizeof(float) * (size_t)B * q_len * h_q * (size_t)w.score_stride;
  return w;
}

// (positions are counted in 32 bits, some steps of a warp past the last one)
static bool mass_sizes_ok(int B, int q_len, int h_q, int h_kv, int d, int mass_len) {
  return B > 0 && q_len > 0 && h_q > 0 && h_kv > 0 && d > 0 && mass_len > 0 && h_q % h_kv == 0 &&
         mass_len <= (1 << 30) && (int64_t)q_len * (h_q / h_kv) <= 16;
}

static tl_status decode_pages(const void* q, const void* k_cache, const void* v_cache,
                              const int32_t* page_table, int32_t n_pages_per_head,
                              const int32_t* page_lens, float* out, int32_t B, int32_t h_q,
                              int32_t h_kv, int32_t d, int32_t num_pages, int32_t page_size,
                              float scale, tl_dtype dtype, void* workspace,
                              size_t workspace_bytes, uint32_t* error_word, void* stream,
                              const float* k_scales, const float* v_scales) {
  DecodeExtra ex;
  ex.head_tables = true;
  return decode_impl<true>(q, k_cache, v_cache, page_table, n_pages_per_head, page_lens, out, B,
                           1, h_q, h_kv, d, num_pages, page_size, 0, 0, scale, dtype, workspace,
                           workspace_bytes, error_word, stream, NewRows(), k_scales, v_scales,
                           ex);
}

static tl_status decode_mass(const void* q, const void* k_cache, const void* v_cache,
                             const int32_t* block_table, int32_t max_pages_per_seq,
                             const int32_t* context_lens, float* out, float* mass,
                             int32_t mass_len, int32_t B, int32_t q_len, int32_t h_q,
                             int32_t h_kv, int32_t d, int32_t num_pages, int32_t page_size,
                             int32_t window, float scale, tl_dtype dtype, void* workspace,
                             size_t workspace_bytes, uint32_t* error_word, void* stream,
                             const float* k_scales, const float* v_scales) {
  if (!mass || !aligned16(mass) || mass_len <= 0) return TL_ERR_INVALID_ARG;
  if (B <= 0 || q_len <= 0 || h_q <= 0 || h_kv <= 0 || d <= 0 || h_q % h_kv)
    return TL_ERR_INVALID_ARG;
  if (!mass_sizes_ok(B, q_len, h_q, h_kv, d, mass_len)) return TL_ERR_UNSUPPORTED;
  const MassWorkspace w = mass_ws_layout(B, q_len, h_q, h_kv, d, mass_len);
  DecodeExtra ex;
  ex.key_cap = mass_len;
  ex.mass = mass;
  ex.mass_len = mass_len;
  ex.score_stride = w.score_stride;
  // a missing, small or misaligned workspace is refused by decode_impl after
  // its other checks: it is told that it has none
  if (workspace_bytes < w.bytes) workspace = nullptr;
  if (workspace) {
    ex.stats = reinterpret_cast<float*>(static_cast<char*>(workspace) + w.stats);
    ex.scores = reinterpret_cast<float*>(static_cast<char*>(workspace) + w.scores);
  }
  return decode_impl<true>(q, k_cache, v_cache, block_table, max_pages_per_seq, context_lens, out,
                           B, q_len, h_q, h_kv, d, num_pages, page_size, window, 0, scale, dtype,
                           workspace, workspace_bytes, error_word, stream, NewRows(), k_scales,
                           v_scales, ex);
}

}  // namespace tl

extern "C" tl_status tl_paged_attn_decode_pages(
    const void* q, const void* k_cache, const void* v_cache, const int32_t* page_table,
    int32_t n_pages_per_head, const int32_t* page_lens, float* out, int32_t B, int32_t h_q,
    int32_t h_kv, int32_t d, int32_t num_pages, int32_t page_size, float scale, tl_dtype dtype,
    void* workspace, size_t workspace_bytes, uint32_t* error_word, void* stream) {
  return tl::decode_pages(q, k_cache, v_cache, page_table, n_pages_per_head, page_lens, out, B,
                          h_q, h_kv, d, num_pages, page_size, scale, dtype, workspace,
                          workspace_bytes, error_word, stream, nullptr, nullptr);
}

extern "C" tl_status tl_paged_attn_decode_pages_int8(
    const void* q, const int8_t* k_codes, const int8_t* v_codes, const float* k_scales,
    const float* v_scales, const int32_t* page_table, int32_t n_pages_per_head,
    const int32_t* page_lens, float* out, int32_t B, int32_t h_q, int32_t h_kv, int32_t d,
    int32_t num_pages, int32_t page_size, float scale, void* workspace, size_t workspace_bytes,
    uint32_t* error_word, void* stream) {
  if (!k_scales || !v_scales) return TL_ERR_INVALID_ARG;
  return tl::decode_pages(q, k_codes, v_codes, page_table, n_pages_per_head, page_lens, out, B,
                          h_q, h_kv, d, num_pages, page_size, scale, TL_FP8_E4M3, workspace,
                          workspace_bytes, error_word, stream, k_scales, v_scales);
}

extern "C" size_t tl_paged_attn_decode_mass_workspace_size(int32_t B, int32_t q_len, int32_t h_q,
                                                           int32_t h_kv, int32_t d,
                                                           int32_t mass_len) {
  if (!tl::mass_sizes_ok(B, q_len, h_q, h_kv, d, mass_len)) return 0;
  return tl::mass_ws_layout(B, q_len, h_q, h_kv, d, mass_len).bytes;
}

extern "C" tl_status tl_paged_attn_decode_mass(
    const void* q, const void* k_cache, const void* v_cache, const int32_t* block_table,
    int32_t max_pages_per_seq, const int32_t* context_lens, float* out, float* mass,
    int32_t mass_len, int32_t B, int32_t q_len, int32_t h_q, int32_t h_kv, int32_t d,
    int32_t num_pages, int32_t page_size, int32_t window, float scale, tl_dtype dtype,
    void* workspace, size_t workspace_bytes, uint32_t* error_word, void* stream) {
  return tl::decode_mass(q, k_cache, v_cache, block_table, max_pages_per_seq, context_lens, out,
                         mass, mass_len, B, q_len, h_q, h_kv, d, num_pages, page_size, window,
                         scale, dtype, workspace, workspace_bytes, error_word, stream, nullptr,
                         nullptr);
}

extern "C" tl_status tl_paged_attn_decode_mass_int8(
    const void* q, const int8_t* k_codes, const int8_t* v_codes, const float* k_scales,
    const float* v_scales, const int32_t* block_table, int32_t max_pages_per_seq,
    const int32_t* context_lens, float* out, float* mass, int32_t mass_len, int32_t B,
    int32_t q_len, int32_t h_q, int32_t h_kv, int32_t d, int32_t num_pages, int32_t page_size,
    int32_t window, float scale, void* workspace, size_t workspace_bytes, uint32_t* error_word,
    void* stream) {
  if (!k_scales || !v_scales) return TL_ERR_INVALID_ARG;
  return tl::decode_mass(q, k_codes, v_codes, block_table, max_pages_per_seq, context_lens, out,
                         mass, mass_len, B, q_len, h_q, h_kv, d, num_pages, page_size, window,
                         scale, TL_FP8_E4M3, workspace, workspace_bytes, error_word, stream,
                         k_scales, v_scales);
}
