// Attention of new tokens over a paged cache: o = sum_j softmax_j(scale q . k_j) v_j.
#include "paged.cuh"

namespace gptq {
namespace paged {
namespace {

// One warp per (row, head): the formula as it stands, one pass with the running maximum and sum.
template <typename T, int D, int BITS>
__global__ void __launch_bounds__(128) rows_kernel(const Args a) {
  const int64_t w = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  const int t = static_cast<int>(w / a.heads), h = static_cast<int>(w % a.heads);
  if (t >= a.tokens) return;
  int lo = 0, hi = a.seqs;  // the last sequence that starts at or before t
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    (__ldg(a.starts + mid) <= t ? lo : hi) = mid;
  }
  const Seq q = sequence(a, lo);
  const int i = t - q.start;
  if (i < 0 || i >= q.n || q.n * a.group <= kStepRows) return;
  float m, l, acc[D / 32];
  row_attention<T, D, BITS>(a, lo, h / a.group, static_cast<const T*>(a.q) + t * a.q_ts + h * a.q_hs, 0, seen(a, q, i),
                            m, l, acc);
  const float inv = l == 0.f ? 0.f : 1.f / l;
  T* o = static_cast<T*>(a.out) + (static_cast<int64_t>(t) * a.heads + h) * D;
#pragma unroll
  for (int c = 0; c < D / 32; ++c) o[lane + 32 * c] = to16<T>(acc[c] * inv);
}

template <typename T, int D>
int launch(const Args& a, int bits, cudaStream_t s) {
  const unsigned grid = static_cast<unsigned>((static_cast<int64_t>(a.tokens) * a.heads + 3) / 4);
  if (bits == 16)
    rows_kernel<T, D, 16><<<grid, 128, 0, s>>>(a);
  else if (bits == 8)
    rows_kernel<T, D, 8><<<grid, 128, 0, s>>>(a);
  else
    rows_kernel<T, D, 4><<<grid, 128, 0, s>>>(a);
  return after_launch();
}

}  // namespace
}  // namespace paged
}  // namespace gptq

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
      tokens * heads > (int64_t(1) << 31))
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
  GPTQ_TRY(paged::run_step(a, dtype, head_dim, bits, s));
  if (static_cast<int64_t>(a.max_q) * a.group <= paged::kStepRows) return GPTQ_OK;
  if (dtype == GPTQ_BF16)
    return head_dim == 128 ? paged::launch<__nv_bfloat16, 128>(a, bits, s) : paged::launch<__nv_bfloat16, 64>(a, bits, s);
  return head_dim == 128 ? paged::launch<__half, 128>(a, bits, s) : paged::launch<__half, 64>(a, bits, s);
}
