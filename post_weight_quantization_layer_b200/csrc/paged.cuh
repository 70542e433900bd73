// What the kernels of the attention over a paged cache share: their arguments, where a key
// lies, and the plain row of the formula.
#pragma once

#include "common.cuh"

namespace gptq {

// kvcache.cu: argument checks of a cache.
int check_cache(const void* kc, const void* vc, const float* ks, const uint8_t* kz, const float* vs, const uint8_t* vz,
                int bits, int64_t pages, int page_size, int kv_heads, int head_dim, int dtype);

namespace paged {

struct Args {
  const void* q;
  void* out;
  const void *kc, *vc;
  const float *ks, *vs;
  const uint8_t *kz, *vz;
  const int32_t *table, *lens, *starts;
  int64_t table_width, q_ts, q_hs;
  int pages, page_shift, tokens, heads, kv_heads, group, seqs, max_q, causal;
  float scale_log2;  // scale * log2(e): scores are taken to base 2
};

struct Seq {
  int start, n, len;  // first row, rows, keys
};

__device__ __forceinline__ Seq sequence(const Args& a, int s) {
  Seq q;
  const int64_t most = min(a.table_width << a.page_shift, int64_t(2147483647));
  q.len = static_cast<int>(max(int64_t(0), min(static_cast<int64_t>(__ldg(a.lens + s)), most)));
  q.start = max(0, min(__ldg(a.starts + s), a.tokens));
  q.n = min(max(min(__ldg(a.starts + s + 1), a.tokens) - q.start, 0), a.max_q);
  return q;
}

// Keys that row i sees (0 .. the count - 1).
__device__ __forceinline__ int seen(const Args& a, const Seq& q, int i) {
  return a.causal ? max(0, min(q.len, q.len - q.n + i + 1)) : q.len;
}

// Vector index of key j of sequence s in [pages, kv_heads, page_size].
__device__ __forceinline__ int64_t key_at(const Args& a, int s, int h, int j) {
  const int id = __ldg(a.table + s * a.table_width + (j >> a.page_shift));
  const int64_t page = min(max(id, 0), a.pages - 1);
  return ((page * a.kv_heads + h) << a.page_shift) + (j & ((1 << a.page_shift) - 1));
}

// Values of a vector: 8 from element c (a multiple of 8), or one.
template <typename T, int D, int BITS>
__device__ __forceinline__ void values8(const void* codes, const float* scales, const uint8_t* zeros, int64_t at, int c,
                                        float (&v)[8]) {
  if constexpr (BITS == 16) {
    const uint4 w = __ldg(reinterpret_cast<const uint4*>(static_cast<const T*>(codes) + at * D + c));
    const T* e = reinterpret_cast<const T*>(&w);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = to_f32(e[i]);
  } else {
    const uint8_t* row = static_cast<const uint8_t*>(codes) + at * (D * BITS / 8) + c * BITS / 8;
    uint32_t w[2];
    if constexpr (BITS == 8)
      *reinterpret_cast<uint2*>(w) = __ldg(reinterpret_cast<const uint2*>(row));
    else
      w[0] = __ldg(reinterpret_cast<const uint32_t*>(row));
    const float s = __ldg(scales + at);
    const int z = __ldg(zeros + at);
#pragma unroll
    for (int i = 0; i < 8; ++i)
      v[i] = s * static_cast<float>(static_cast<int>((w[i * BITS / 32] >> (i * BITS % 32)) & ((1u << BITS) - 1u)) - z);
  }
}
template <typename T, int D, int BITS>
__device__ __forceinline__ float value1(const void* codes, const float* scales, const uint8_t* zeros, int64_t at, int c) {
  if constexpr (BITS == 16) {
    return to_f32(__ldg(static_cast<const T*>(codes) + at * D + c));
  } else {
    const int w = __ldg(static_cast<const uint8_t*>(codes) + at * (D * BITS / 8) + c * BITS / 8);
    const int q = (w >> (c * BITS % 8)) & ((1 << BITS) - 1);
    return __ldg(scales + at) * static_cast<float>(q - __ldg(zeros + at));
  }
}

// One row over the keys k0 .. k1-1, by one warp, in fp32: running maximum m (base 2), sum l and
// the weighted sum of the lane's values lane, lane + 32, ...  32 keys at a time: a key per lane
// for the scores, then all lanes on one key's values after another.  Keys outside the range are
// never read.
template <typename T, int D, int BITS>
__device__ void row_attention(const Args& a, int s, int h, const T* qrow, int k0, int k1, float& m, float& l,
                              float (&acc)[D / 32]) {
  const int lane = threadIdx.x & 31;
  m = -INFINITY;
  l = 0.f;
#pragma unroll
  for (int c = 0; c < D / 32; ++c) acc[c] = 0.f;
  for (int base = k0; base < k1; base += 32) {
    const int j = base + lane;
    float sc = -INFINITY;
    int64_t at = 0;
    if (j < k1) {
      at = key_at(a, s, h, j);
      float dot = 0.f;
      for (int c = 0; c < D; c += 8) {
        float kv[8];
        values8<T, D, BITS>(a.kc, a.ks, a.kz, at, c, kv);
#pragma unroll
        for (int i = 0; i < 8; ++i) dot = fmaf(to_f32(qrow[c + i]), kv[i], dot);
      }
      sc = dot * a.scale_log2;
    }
    float mx = sc;
    for (int o = 16; o; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    mx = fmaxf(m, mx);
    const float ref = mx == -INFINITY ? 0.f : mx;
    const float p = j < k1 ? exp2f(sc - ref) : 0.f;
    const float corr = exp2f(m - ref);
    float sum = p;
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    l = l * corr + sum;
    m = mx;
#pragma unroll
    for (int c = 0; c < D / 32; ++c) acc[c] *= corr;
    for (int i = 0; i < min(32, k1 - base); ++i) {
      const float pi = __shfl_sync(0xffffffffu, p, i);
      const int64_t ai = __shfl_sync(0xffffffffu, at, i);
#pragma unroll
      for (int c = 0; c < D / 32; ++c)
        acc[c] = fmaf(pi, value1<T, D, BITS>(a.vc, a.vs, a.vz, ai, lane + 32 * c), acc[c]);
    }
  }
}

template <typename T>
__device__ __forceinline__ T to16(float v);
template <>
__device__ __forceinline__ __half to16<__half>(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ __nv_bfloat16 to16<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// The launches of one call overlap: each may start, and work out its share, while the one before it
// drains, and waits for it before it reads what it wrote, or else before it ends, so that the end of the
// last launch is the end of all.
__device__ __forceinline__ void next_may_start() { asm volatile("griddepcontrol.launch_dependents;"); }
__device__ __forceinline__ void wait_for_last() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

template <typename... P, typename... A>
int launch_next(void (*kernel)(P...), dim3 grid, int threads, int smem, cudaStream_t s, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...) != cudaSuccess) {
    cudaGetLastError();
    return GPTQ_ERR_CUDA;
  }
  return after_launch();
}

// An item (the rows of a sequence and kv head, or a tile of them) that the border before share c cuts; told by
// CTA c where no earlier border cuts the same item.  Its parts lie in the first slots of the CTAs c0 + 1 .. c1
// and in slot `slot0` of c0 (a CTA's first piece is in its slot 0, its last in slot 1).
struct Cut {
  int c0, c1, slot0;  // c1 < 0: nothing to join
  int start, n, head, tile;
};

// The cut at a CTA's first piece, which begins `skipped` units inside its item of `units`.
__device__ __forceinline__ Cut cut_at(int64_t at, int64_t per, int skipped, int units, const Seq& q, int head, int tile) {
  Cut c{0, -1, 0, q.start, q.n, head, tile};
  if (skipped > 0) {
    const int64_t begin = at - skipped;
    c.c0 = static_cast<int>(begin / per);
    c.slot0 = begin == c.c0 * per ? 0 : 1;
    if (c.c0 + 1 == static_cast<int>(blockIdx.x)) c.c1 = static_cast<int>((begin + units - 1) / per);
  }
  return c;
}

// paged_step.cu: the sequences with 1 .. 16 rows (tokens x heads of a kv head).  step_grid: CTAs, and how many take
// an item together (0: items are cut; a part of a cut item is step_part(head_dim) floats).
constexpr int kStepRows = 16;
__host__ __device__ constexpr int step_part(int d) { return kStepRows * (d + 2); }
int step_grid(const Args& a, int* team);
int run_step(const Args& a, int dtype, int head_dim, int bits, int grid, int team, float* part, Cut* cut, cudaStream_t s);

// paged_chunk.cu: the sequences with more rows, in tiles of kTileRows.  odd: a word per CTA, not 0 where it met
// a result that is not finite.  `next`: follows a launch of the same call.
constexpr int kTileRows = 256;
__host__ __device__ constexpr int chunk_part(int d) { return kTileRows * (d + 2); }
int run_chunk(const Args& a, int dtype, int head_dim, int bits, int grid, float* part, Cut* cut, int* odd, bool next,
              cudaStream_t s);
int run_chunk_redo(const Args& a, int dtype, int head_dim, int bits, const int* odd, int n, cudaStream_t s);
int chunk_device_status(int clear);

}  // namespace paged
}  // namespace gptq
