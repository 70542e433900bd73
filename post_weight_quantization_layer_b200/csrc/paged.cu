// Attention of new tokens over a paged cache: o = sum_j softmax_j(scale q . k_j) v_j.  Arguments are
// checked here; sequences with at most kStepRows rows (tokens x heads of a kv head) go to the kernel
// of paged_step.cu, the others to that of paged_chunk.cu, each sequence by its own number of rows on
// the device.
// The parts that the two kernels leave behind where their shares cut an item are joined by one launch.
#include "paged.cuh"

namespace gptq {
namespace paged {
namespace {

constexpr int JN_THREADS = kTileRows;

__device__ __forceinline__ float pow2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// out = sum_x 2^(m_x - m) o_x / sum_x 2^(m_x - m) l_x over the parts of an item, in their order.  Borders of
// the step kernel: a CTA each, 4 columns of a row per thread; borders of the chunk kernel: D/8 CTAs each, 8
// columns of a row per thread (its parts lie column by column).
template <typename T, int D>
__global__ void __launch_bounds__(JN_THREADS) join_kernel(const Args a, const float* __restrict__ step,
                                                          const Cut* __restrict__ step_cut, int step_n,
                                                          const float* __restrict__ chunk,
                                                          const Cut* __restrict__ chunk_cut) {
  next_may_start();
  wait_for_last();
  const int b = blockIdx.x;
  const bool steps = b < step_n;
  const int border = steps ? b : (b - step_n) / (D / 8);
  const Cut c = (steps ? step_cut : chunk_cut)[border + 1];
  if (c.c1 < 0) return;
  if (steps) {
    const int rows = c.n * a.group;
    for (int e = threadIdx.x; e < rows * (D / 4); e += JN_THREADS) {
      const int row = e / (D / 4), col = (e % (D / 4)) * 4;
      float m = -INFINITY, l = 0.f;
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
      for (int x = c.c0; x <= c.c1; ++x) {
        const float* p = step + (2 * static_cast<int64_t>(x) + (x == c.c0 ? c.slot0 : 0)) * step_part(D);
        const float pm = p[kStepRows * D + row], pl = p[kStepRows * (D + 1) + row];
        const float4 y = *reinterpret_cast<const float4*>(p + row * D + col);
        const float mm = fmaxf(m, pm), ref = mm == -INFINITY ? 0.f : mm;
        const float f0 = pow2(m - ref), f1 = pow2(pm - ref);
        m = mm;
        l = l * f0 + pl * f1;
        v.x = v.x * f0 + y.x * f1;
        v.y = v.y * f0 + y.y * f1;
        v.z = v.z * f0 + y.z * f1;
        v.w = v.w * f0 + y.w * f1;
      }
      const float inv = l == 0.f ? 0.f : 1.f / l;
      const int i = row / a.group;
      T* dst = static_cast<T*>(a.out) +
               ((static_cast<int64_t>(c.start) + i) * a.heads + c.head * a.group + (row - i * a.group)) * D + col;
      alignas(8) T o[4] = {to16<T>(v.x * inv), to16<T>(v.y * inv), to16<T>(v.z * inv), to16<T>(v.w * inv)};
      *reinterpret_cast<uint2*>(dst) = *reinterpret_cast<const uint2*>(o);
    }
    return;
  }
  const int r = threadIdx.x, col = (b - step_n) % (D / 8) * 8;
  const int row = c.tile * kTileRows + r;
  if (row >= c.n * a.group) return;
  float m = -INFINITY, l = 0.f, v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = 0.f;
  for (int x = c.c0; x <= c.c1; ++x) {
    const float* p = chunk + (2 * static_cast<int64_t>(x) + (x == c.c0 ? c.slot0 : 0)) * chunk_part(D);
    const float pm = p[D * kTileRows + r], pl = p[(D + 1) * kTileRows + r];
    float y[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = p[(col + i) * kTileRows + r];
    const float mm = fmaxf(m, pm), ref = mm == -INFINITY ? 0.f : mm;
    const float f0 = pow2(m - ref), f1 = pow2(pm - ref);
    m = mm;
    l = l * f0 + pl * f1;
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = v[i] * f0 + y[i] * f1;
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  const int i = row / a.group;
  T* dst = static_cast<T*>(a.out) +
           ((static_cast<int64_t>(c.start) + i) * a.heads + c.head * a.group + (row - i * a.group)) * D + col;
  alignas(16) T o[8];
#pragma unroll
  for (int x = 0; x < 8; ++x) o[x] = to16<T>(v[x] * inv);
  *reinterpret_cast<uint4*>(dst) = *reinterpret_cast<const uint4*>(o);
}

// Launches of one call: sequences with few rows, sequences with more, the join, the second look at results
// that are not finite; each may start while the one before it drains.
int attend(const Args& a, int dtype, int head_dim, int bits, cudaStream_t s) {
  const bool chunks = static_cast<int64_t>(a.max_q) * a.group > kStepRows;
  const bool steps = a.group <= kStepRows;  // sequences with few rows may be among long ones
  int team = 1;
  const int step_ctas = steps ? step_grid(a, &team) : 0;
  const int step_n = team == 0 ? step_ctas : 0, chunk_n = chunks ? num_sms() : 0;
  const size_t step_bytes = static_cast<size_t>(step_n) * (2 * step_part(head_dim) * sizeof(float) + sizeof(Cut));
  const size_t chunk_bytes =
      static_cast<size_t>(chunk_n) * (2 * chunk_part(head_dim) * sizeof(float) + sizeof(Cut) + sizeof(int));
  void* work = nullptr;
  if (step_bytes + chunk_bytes) GPTQ_TRY(pool_alloc(&work, step_bytes + chunk_bytes, s));
  float* chunk_parts = static_cast<float*>(work);
  float* step_parts = chunk_parts + static_cast<size_t>(chunk_n) * 2 * chunk_part(head_dim);
  Cut* chunk_cut = reinterpret_cast<Cut*>(step_parts + static_cast<size_t>(step_n) * 2 * step_part(head_dim));
  Cut* step_cut = chunk_cut + chunk_n;
  int* odd = reinterpret_cast<int*>(step_cut + step_n);
  int st = GPTQ_OK;
  if (steps) st = run_step(a, dtype, head_dim, bits, step_ctas, team, step_parts, step_cut, s);
  if (st == GPTQ_OK && chunks)
    st = run_chunk(a, dtype, head_dim, bits, chunk_n, chunk_parts, chunk_cut, odd, steps, s);
  const int step_borders = step_n > 1 ? step_n - 1 : 0, chunk_borders = chunk_n > 1 ? chunk_n - 1 : 0;
  const dim3 joins(static_cast<unsigned>(step_borders + chunk_borders * (head_dim / 8)));
  if (st == GPTQ_OK && joins.x) {
#define GPTQ_JOIN(T, D)                                                                                     \
  launch_next(join_kernel<T, D>, joins, JN_THREADS, 0, s, a, static_cast<const float*>(step_parts),          \
              static_cast<const Cut*>(step_cut), step_borders, static_cast<const float*>(chunk_parts),       \
              static_cast<const Cut*>(chunk_cut))
    if (dtype == GPTQ_BF16)
      st = head_dim == 128 ? GPTQ_JOIN(__nv_bfloat16, 128) : GPTQ_JOIN(__nv_bfloat16, 64);
    else
      st = head_dim == 128 ? GPTQ_JOIN(__half, 128) : GPTQ_JOIN(__half, 64);
#undef GPTQ_JOIN
  }
  if (st == GPTQ_OK && chunks) st = run_chunk_redo(a, dtype, head_dim, bits, odd, chunk_n, s);
  if (work) pool_free(work, s);
  return st;
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
  if (work && out == q) return GPTQ_ERR_INVALID_ARG;  // rows are read again after others are written
  if (heads % kv_heads || !(scale > 0.f && scale < INFINITY)) return GPTQ_ERR_INVALID_ARG;
  if (heads / kv_heads > 64 || heads > 65535 || seqs > (1 << 20) || table_width > (int64_t(1) << 27) ||
      table_width * page_size > (int64_t(1) << 31) - 1024 ||
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
  return paged::attend(a, dtype, head_dim, bits, s);
}
