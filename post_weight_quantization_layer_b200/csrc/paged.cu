// Attention of new tokens over a paged cache: o = sum_j softmax_j(scale q . k_j) v_j.  Arguments are
// checked here; sequences with at most kStepRows rows (tokens x heads of a kv head) go to the kernel
// of paged_step.cu, the others to that of paged_chunk.cu, each sequence by its own number of rows on
// the device.
#include "paged.cuh"

using namespace gptq;

extern "C" int gptq_paged_attention(const void* q, int dtype, int64_t tokens, int heads, int kv_heads, int head_dim,
                                    int64_t q_token_stride, int64_t q_head_stride, const void* k_cache,
                                    const void* v_cache, const float* k_scales, const uint8_t* k_zeros,
                                    const float* v_scales, const uint8_t* v_zeros, int bits, int64_t pages,
                                    int page_size, const int32_t* page_table, int64_t table_width,
                                    const int32_t* kv_lens, const int32_t* q_starts, int64_t seqs, int64_t max_q_len,
                                    int causal, float scale, void* out, void* stream) {
  if (tokens < 0 || seqs < 0 || heads <= 0 || max_q_len < 0) return GPTQ_ERR_INVALID_ARG;
  const bool work = tokens > 0 && seqs > 0 && max_q_len > 0;
  if (work && (!q || !out || !page_table || !kv_lens || !q_starts || table_width <= 0)) return GPTQ_ERR_INVALID_ARG;
  GPTQ_TRY(check_cache(k_cache, v_cache, k_scales, k_zeros, v_scales, v_zeros, bits, pages, page_size, kv_heads,
                       head_dim, dtype));
  if (heads % kv_heads || !(scale > 0.f && scale < INFINITY)) return GPTQ_ERR_INVALID_ARG;
  if (heads / kv_heads > 64 || heads > 65535 || seqs > (1 << 20) || table_width > (int64_t(1) << 27) ||
      tokens * heads > (int64_t(1) << 30))
    return GPTQ_ERR_UNSUPPORTED;
  if (((q_token_stride | q_head_stride) & 7) || !aligned16(q) || !aligned16(out)) return GPTQ_ERR_UNSUPPORTED;
  if (!work) return GPTQ_OK;
  paged::Args a;
  a.q = q;
  a.out = out;
  a.kc = k_cache;
  a.vc = v_cache;
  a.ks = k_scales;
  a.vs = v_scales;
  a.kz = k_zeros;
  a.vz = v_zeros;
  a.table = page_table;
  a.lens = kv_lens;
  a.starts = q_starts;
  a.table_width = table_width;
  a.q_ts = q_token_stride;
  a.q_hs = q_head_stride;
  a.pages = static_cast<int>(pages);
  a.page_shift = 0;
  while ((1 << a.page_shift) < page_size) ++a.page_shift;
  a.tokens = static_cast<int>(tokens);
  a.heads = heads;
  a.kv_heads = kv_heads;
  a.group = heads / kv_heads;
  a.seqs = static_cast<int>(seqs);
  a.max_q = static_cast<int>(max_q_len < tokens ? max_q_len : tokens);
  a.causal = causal != 0;
  a.scale_log2 = scale * 1.4426950408889634f;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool chunks = static_cast<int64_t>(a.max_q) * a.group > paged::kStepRows;
  if (chunks) GPTQ_TRY(paged::run_chunk(a, dtype, head_dim, bits, s));
  // sequences with few rows may be among long ones; there are none where a single row is more
  if (a.group > paged::kStepRows) return GPTQ_OK;
  return paged::run_step(a, dtype, head_dim, bits, chunks, s);
}
