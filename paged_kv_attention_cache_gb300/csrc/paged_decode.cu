// The decode entry points of the C ABI; the kernels and their launch are in
// paged_decode.cuh.
#include "paged_decode.cuh"

namespace tl {

// The plan launch of a step that rotates its queries and new keys itself: beside
// the plan, CTAs that rotate the queries into the workspace, where the attention
// kernel reads them, and write the rows: one warp per pass over a token's heads
// in rotary units, or per row where rows are not made of them.  Measured, 32
// query and 8 KV heads of 128: a step of 64 sequences of 2,048 keys takes 88.6
// us (tl_paged_attn_decode_write of rotated rows 89.3, the append and the decode
// in two calls 92.2), of one of 1,024 17.6 us (18.0, 20.5); e4m3 pools 55.2
// (55.5, 58.1) and 17.5, int8 60.6 (60.5, 64.5) and 20.2, f32 1122 (1122, 1127)
// and 35.6.
template <bool F32, int KIND, bool INTER>
struct TurnedRows {
  RopeRows R;
  int units;  // of a row; 0: element by element
  __device__ __forceinline__ void write(const DecodeParams& P) const {
    __shared__ float4 cs[32][4 * kRopeStepUnits];
    const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
    const int warps = P.B <= kWarpPlanMax ? kWriteWarps : (int)(blockDim.x >> 5);
    if (wid >= warps) return;
    const int heads = R.h_q + 2 * R.h_kv, HW = units ? 32 / units : 1;
    const int per = (heads + HW - 1) / HW;
    const int64_t stride = (int64_t)(gridDim.x - 1) * warps;
    for (int64_t i = (int64_t)(blockIdx.x - 1) * warps + wid; i < (int64_t)R.n * per;
         i += stride) {
      const int64_t t = i / per;
      const int h = (int)(i - t * per) * HW;
      if (units) rope_units<F32, KIND, INTER, 1>(R, t, h, heads, units, HW, lane, cs[wid]);
      else rope_row<F32, KIND>(R, t, h, lane);
    }
  }
};

cudaError_t launch_plan_rope(const DecodeParams& P, const RopeStep& r, int plan_threads,
                             int target_splits, int first_dynamic, bool f32, cudaStream_t st) {
  const RopeRows& R = r.rows;
  const bool inter = R.interleaved != 0;
  const int heads = R.h_q + 2 * R.h_kv, HW = r.units ? 32 / r.units : 1;
  const int64_t warps = (int64_t)R.n * ((heads + HW - 1) / HW);
  const int wpc = P.B <= kWarpPlanMax ? kWriteWarps : plan_threads / 32;
  const unsigned grid = 1 + (unsigned)std::min<int64_t>(num_sms(), (warps + wpc - 1) / wpc);
#define TL_PLAN_ROPE(F32, K, I)                          \
  decode_plan_kernel<false, TurnedRows<F32, K, I>>       \
      <<<grid, plan_threads, 0, st>>>(P, target_splits, first_dynamic, {R, r.units})
  if (f32 && inter) TL_PLAN_ROPE(true, kRopeSame, true);
  else if (f32) TL_PLAN_ROPE(true, kRopeSame, false);
  else if (r.kind == kRopeSame && inter) TL_PLAN_ROPE(false, kRopeSame, true);
  else if (r.kind == kRopeSame) TL_PLAN_ROPE(false, kRopeSame, false);
  else if (r.kind == kRopeE4m3 && inter) TL_PLAN_ROPE(false, kRopeE4m3, true);
  else if (r.kind == kRopeE4m3) TL_PLAN_ROPE(false, kRopeE4m3, false);
  else if (inter) TL_PLAN_ROPE(false, kRopeInt8, true);
  else TL_PLAN_ROPE(false, kRopeInt8, false);
#undef TL_PLAN_ROPE
  return cudaGetLastError();
}

// Workspace of a step that rotates: the decode's, then the rotated queries (of
// up to 4 bytes an element).
static size_t rope_ws_queries(int32_t B, int32_t h_q, int32_t h_kv, int32_t d) {
  return align_up(decode_ws_layout(B, h_q, h_kv, d, nullptr, nullptr), 256);
}

static tl_status decode_write_rope(
    const void* q, int64_t q_stride, const void* k_new, int64_t k_stride, const void* v_new,
    int64_t v_stride, const int64_t* slot_mapping, const int32_t* positions,
    const uint64_t* freqs, int32_t rot_dim, int32_t interleaved, float rope_scale, void* k_cache,
    void* v_cache, float* k_scales, float* v_scales, const int32_t* block_table,
    int32_t max_pages_per_seq, const int32_t* context_lens, float* out, int32_t B, int32_t h_q,
    int32_t h_kv, int32_t d, int32_t num_pages, int32_t page_size, int32_t window,
    int32_t ring_pages, float scale, tl_dtype dtype, void* workspace, size_t workspace_bytes,
    uint32_t* error_word, void* stream) {
  if (B <= 0 || h_q <= 0 || h_kv <= 0 || d <= 0 || num_pages <= 0 || page_size <= 0 ||
      h_q % h_kv || !q)
    return TL_ERR_INVALID_ARG;
  if (dtype != TL_BF16 && dtype != TL_F32 && dtype != TL_FP8_E4M3 && dtype != TL_INT8)
    return TL_ERR_UNSUPPORTED;
  if (d > 16 * kRopeStepUnits) return TL_ERR_UNSUPPORTED;
  const tl_dtype q_dtype = dtype == TL_F32 ? TL_F32 : TL_BF16;
  const size_t queries = rope_ws_queries(B, h_q, h_kv, d);
  const size_t need = queries + sizeof(float) * (size_t)B * h_q * d;
  // a missing, small or misaligned workspace is refused by decode_impl after
  // its other checks: it is told that it has none
  if (workspace_bytes < need || (reinterpret_cast<uintptr_t>(workspace) & 255u))
    workspace = nullptr;
  if (!aligned_to(q, q_dtype == TL_F32 ? 4 : 2) || q_stride < 0) return TL_ERR_INVALID_ARG;
  void* q_out = workspace ? static_cast<char*>(workspace) + queries : nullptr;
  RopeStep step;
  const tl_status ok = rope_rows_checked(
      workspace ? q : nullptr, q_stride, q_out, (int64_t)h_q * d, k_new, k_stride, v_new,
      v_stride, q_dtype, k_cache, v_cache, k_scales, v_scales, slot_mapping, positions, freqs,
      rot_dim, interleaved, rope_scale, B, num_pages, page_size, workspace ? h_q : 0, h_kv, d,
      dtype, error_word, &step.rows, &step.kind);
  if (ok != TL_OK) return ok;
  // the plan writes the workspace beside the CTAs that read the rows
  const int64_t row = (int64_t)h_kv * d;
  const size_t pool = (size_t)num_pages * page_size * row *
                      (dtype == TL_F32 ? 4 : dtype == TL_BF16 ? 2 : 1);
  const int elem = q_dtype == TL_F32 ? 4 : 2;
  const struct {
    const void* p;
    size_t bytes;
  } spans[] = {{q, (size_t)((B - 1) * q_stride + (int64_t)h_q * d) * elem},
               {k_new, (size_t)((B - 1) * k_stride + row) * elem},
               {v_new, (size_t)((B - 1) * v_stride + row) * elem},
               {k_cache, pool},
               {v_cache, pool},
               {k_scales, k_scales ? pool / d * sizeof(float) : 0},
               {v_scales, v_scales ? pool / d * sizeof(float) : 0}};
  for (const auto& s : spans)
    if (workspace && s.bytes && overlap(workspace, need, s.p, s.bytes))
      return TL_ERR_INVALID_ARG;
  if (workspace && over_rope_lists(workspace, need, slot_mapping, positions, freqs, B, rot_dim))
    return TL_ERR_INVALID_ARG;
  step.units = rope_unit_width(step.rows, elem) == 16 / elem ? d / 16 : 0;
  // (q_out stands for q: 256-byte aligned, where q need not be)
  return decode_impl<false>(workspace ? q_out : k_cache, k_cache, v_cache, block_table,
                            max_pages_per_seq, context_lens, out, B, 1, h_q, h_kv, d, num_pages,
                            page_size, window, ring_pages, scale,
                            dtype == TL_INT8 ? TL_FP8_E4M3 : dtype, workspace, workspace_bytes,
                            error_word, stream, NewRows(), k_scales, v_scales, DecodeExtra(),
                            &step);
}

}  // namespace tl

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

extern "C" size_t tl_paged_attn_decode_write_rope_workspace_size(int32_t B, int32_t h_q,
                                                                 int32_t h_kv, int32_t d) {
  if (B <= 0 || h_q <= 0 || h_kv <= 0 || d <= 0 || h_q % h_kv) return 0;
  return tl::rope_ws_queries(B, h_q, h_kv, d) + sizeof(float) * (size_t)B * h_q * d;
}

extern "C" tl_status tl_paged_attn_decode_write_rope(
    const void* q, int64_t q_stride, const void* k_new, int64_t k_stride, const void* v_new,
    int64_t v_stride, const int64_t* slot_mapping, const int32_t* positions,
    const uint64_t* freqs, int32_t rot_dim, int32_t interleaved, float rope_scale, void* k_cache,
    void* v_cache, const int32_t* block_table, int32_t max_pages_per_seq,
    const int32_t* context_lens, float* out, int32_t B, int32_t h_q, int32_t h_kv, int32_t d,
    int32_t num_pages, int32_t page_size, int32_t window, float scale, tl_dtype dtype,
    void* workspace, size_t workspace_bytes, uint32_t* error_word, void* stream) {
  if (dtype == TL_INT8) return TL_ERR_UNSUPPORTED;
  return tl::decode_write_rope(q, q_stride, k_new, k_stride, v_new, v_stride, slot_mapping,
                               positions, freqs, rot_dim, interleaved, rope_scale, k_cache,
                               v_cache, nullptr, nullptr, block_table, max_pages_per_seq,
                               context_lens, out, B, h_q, h_kv, d, num_pages, page_size, window,
                               0, scale, dtype, workspace, workspace_bytes, error_word, stream);
}

extern "C" tl_status tl_paged_attn_decode_write_rope_int8(
    const void* q, int64_t q_stride, const void* k_new, int64_t k_stride, const void* v_new,
    int64_t v_stride, const int64_t* slot_mapping, const int32_t* positions,
    const uint64_t* freqs, int32_t rot_dim, int32_t interleaved, float rope_scale,
    int8_t* k_codes, int8_t* v_codes, float* k_scales, float* v_scales,
    const int32_t* block_table, int32_t max_pages_per_seq, const int32_t* context_lens,
    float* out, int32_t B, int32_t h_q, int32_t h_kv, int32_t d, int32_t num_pages,
    int32_t page_size, int32_t window, float scale, void* workspace, size_t workspace_bytes,
    uint32_t* error_word, void* stream) {
  if (!k_scales || !v_scales) return TL_ERR_INVALID_ARG;
  return tl::decode_write_rope(q, q_stride, k_new, k_stride, v_new, v_stride, slot_mapping,
                               positions, freqs, rot_dim, interleaved, rope_scale, k_codes,
                               v_codes, k_scales, v_scales, block_table, max_pages_per_seq,
                               context_lens, out, B, h_q, h_kv, d, num_pages, page_size, window,
                               0, scale, TL_INT8, workspace, workspace_bytes, error_word,
                               stream);
}

extern "C" tl_status tl_paged_attn_decode_write_rope_ring(
    const void* q, int64_t q_stride, const void* k_new, int64_t k_stride, const void* v_new,
    int64_t v_stride, const int64_t* slot_mapping, const int32_t* positions,
    const uint64_t* freqs, int32_t rot_dim, int32_t interleaved, float rope_scale, void* k_cache,
    void* v_cache, const int32_t* block_table, int32_t max_pages_per_seq,
    const int32_t* context_lens, float* out, int32_t B, int32_t h_q, int32_t h_kv, int32_t d,
    int32_t num_pages, int32_t page_size, int32_t window, int32_t ring_pages, float scale,
    tl_dtype dtype, void* workspace, size_t workspace_bytes, uint32_t* error_word,
    void* stream) {
  if (ring_pages <= 0 || ring_pages > max_pages_per_seq || window <= 0 || page_size <= 0 ||
      (int64_t)ring_pages * page_size < window)
    return TL_ERR_INVALID_ARG;
  if (dtype == TL_INT8) return TL_ERR_UNSUPPORTED;
  return tl::decode_write_rope(q, q_stride, k_new, k_stride, v_new, v_stride, slot_mapping,
                               positions, freqs, rot_dim, interleaved, rope_scale, k_cache,
                               v_cache, nullptr, nullptr, block_table, max_pages_per_seq,
                               context_lens, out, B, h_q, h_kv, d, num_pages, page_size, window,
                               ring_pages, scale, dtype, workspace, workspace_bytes, error_word,
                               stream);
}
