// A paged key/value cache: quantizing vectors as they are written, and reading them back.
//
// One vector (a token's key or value of one kv head, D = 64 or 128 values) is one group of the
// library's uniform quantizer: scale = (hi - lo) / maxq over a range that holds 0, an integer
// zero point, value = scale * (code - zero).  The code is the one nearest to the exact quotient
// x / s (half to even): k = rint(x * (1/s)) is at most one off, and the remainder
// x - k s, which one fused multiply-add gives exactly, settles it against s / 2.  So the codes
// do not depend on how a division rounds.
//
// Both directions are bound by memory.  A vector is D/8 neighbouring threads with 8 values (16
// bytes) each: its range is a shuffle over them, and the codes leave as 8 or 4 bytes per
// thread.  Keys and values go in one launch.
#include <algorithm>

#include "common.cuh"

namespace gptq {
namespace {

constexpr int KC_THREADS = 256;

struct CacheArgs {
  const void *k, *v;  // write: inputs
  void *ko, *vo;      // read: outputs
  int64_t k_ts, k_hs, v_ts, v_hs;
  void *kc, *vc;
  float *ks, *vs;
  uint8_t *kz, *vz;
  int64_t count, slots_total;
  int heads, page_shift;
  const int32_t* slots;
};

template <typename T>
__device__ __forceinline__ T kc16(float v);
template <>
__device__ __forceinline__ __half kc16<__half>(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ __nv_bfloat16 kc16<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// rint of the exact quotient x / s, |x| <= 255 s, s > 0; inv ~ 1/s within two roundings.
__device__ __forceinline__ float rint_quotient(float x, float s, float inv) {
  float k = rintf(x * inv);
  const float e = fmaf(-k, s, x);  // exact: a multiple of the last place of s or of x, below 2 s
  const float a = fabsf(e), h = 0.5f * s;
  const bool odd = (static_cast<int>(k) & 1) != 0;
  if (a > h || (a == h && odd)) k += copysignf(1.f, e);
  return k;
}

// Offset (in vectors) of slot s, head h in [pages, heads, page_size]; -1 outside the cache.
__device__ __forceinline__ int64_t vector_at(const CacheArgs& p, int slot, int h) {
  if (slot < 0 || slot >= p.slots_total) return -1;
  const int64_t page = slot >> p.page_shift;
  return ((page * p.heads + h) << p.page_shift) + (slot & ((1 << p.page_shift) - 1));
}

template <typename T, int D, int BITS>
__global__ void __launch_bounds__(KC_THREADS) cache_write_kernel(const CacheArgs p) {
  constexpr int LPV = D / 8;  // threads of a vector
  const int64_t e = static_cast<int64_t>(blockIdx.x) * KC_THREADS + threadIdx.x;
  const int64_t vec = e / LPV;
  const int l = static_cast<int>(e % LPV);
  // (token, side, head): whole groups of LPV threads (which never cross a warp) leave together
  const int64_t per = 2 * p.heads;
  const int64_t t = vec / per;
  const int sh = static_cast<int>(vec - t * per);
  const bool isv = sh >= p.heads;
  const int h = isv ? sh - p.heads : sh;
  const int64_t at = t < p.count ? vector_at(p, __ldg(p.slots + t), h) : -1;
  uint4 raw = make_uint4(0, 0, 0, 0);
  if (at >= 0)
    raw = *reinterpret_cast<const uint4*>(static_cast<const T*>(isv ? p.v : p.k) + t * (isv ? p.v_ts : p.k_ts) +
                                          h * (isv ? p.v_hs : p.k_hs) + l * 8);
  if constexpr (BITS == 16) {
    if (at >= 0) *reinterpret_cast<uint4*>(static_cast<T*>(isv ? p.vc : p.kc) + at * D + l * 8) = raw;
  } else {
    constexpr float MAXQ = static_cast<float>((1 << BITS) - 1);
    float x[8];
    const T* r = reinterpret_cast<const T*>(&raw);
    float lo = 0.f, hi = 0.f, bad = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      x[i] = to_f32(r[i]);
      lo = fminf(lo, x[i]);
      hi = fmaxf(hi, x[i]);
      bad += x[i] * 0.f;  // NaN as soon as one value is NaN or infinite
    }
#pragma unroll
    for (int o = LPV / 2; o; o >>= 1) {
      lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
      hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
      bad += __shfl_xor_sync(0xffffffffu, bad, o);
    }
    if (at < 0) return;
    if (lo == 0.f && hi == 0.f) {
      lo = -1.f;
      hi = 1.f;
    }
    float s = __fdiv_rn(hi - lo, MAXQ);
    uint32_t code[8];
    uint32_t zero = 0;
    if (bad == 0.f && s < INFINITY) {
      // tiny scales are brought up by a power of two (exactly), where 1/s is finite
      const float up = s < 0x1p-100f ? 0x1p64f : 1.f;
      const float su = s * up, inv = __fdiv_rn(1.f, su);
      const float z = fminf(fmaxf(rint_quotient(-lo * up, su, inv), 0.f), MAXQ);
#pragma unroll
      for (int i = 0; i < 8; ++i)
        code[i] = static_cast<uint32_t>(fminf(fmaxf(rint_quotient(x[i] * up, su, inv) + z, 0.f), MAXQ));
      zero = static_cast<uint32_t>(z);
    } else {
      s = __int_as_float(0x7fc00000);
#pragma unroll
      for (int i = 0; i < 8; ++i) code[i] = 0;
    }
    uint8_t* row = static_cast<uint8_t*>(isv ? p.vc : p.kc) + at * (D * BITS / 8);
    if constexpr (BITS == 8) {
      uint2 w;
      w.x = code[0] | code[1] << 8 | code[2] << 16 | code[3] << 24;
      w.y = code[4] | code[5] << 8 | code[6] << 16 | code[7] << 24;
      *reinterpret_cast<uint2*>(row + l * 8) = w;
    } else {
      uint32_t w = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) w |= code[i] << (4 * i);
      *reinterpret_cast<uint32_t*>(row + l * 4) = w;
    }
    if (l == 0) {
      (isv ? p.vs : p.ks)[at] = s;
      (isv ? p.vz : p.kz)[at] = static_cast<uint8_t>(zero);
    }
  }
}

template <typename T, int D, int BITS>
__global__ void __launch_bounds__(KC_THREADS) cache_read_kernel(const CacheArgs p) {
  constexpr int LPV = D / 8;
  const int64_t e = static_cast<int64_t>(blockIdx.x) * KC_THREADS + threadIdx.x;
  const int64_t vec = e / LPV;
  const int l = static_cast<int>(e % LPV);
  const int64_t per = 2 * p.heads;
  const int64_t t = vec / per;
  if (t >= p.count) return;
  const int sh = static_cast<int>(vec - t * per);
  const bool isv = sh >= p.heads;
  const int h = isv ? sh - p.heads : sh;
  const int64_t at = vector_at(p, __ldg(p.slots + t), h);
  alignas(16) T out[8];
  if (at < 0) {
#pragma unroll
    for (int i = 0; i < 8; ++i) out[i] = kc16<T>(0.f);
  } else if constexpr (BITS == 16) {
    *reinterpret_cast<uint4*>(out) =
        __ldg(reinterpret_cast<const uint4*>(static_cast<const T*>(isv ? p.vc : p.kc) + at * D + l * 8));
  } else {
    const uint8_t* row = static_cast<const uint8_t*>(isv ? p.vc : p.kc) + at * (D * BITS / 8);
    const float s = __ldg((isv ? p.vs : p.ks) + at);
    const int z = __ldg((isv ? p.vz : p.kz) + at);
    uint32_t w[2];
    if constexpr (BITS == 8)
      *reinterpret_cast<uint2*>(w) = __ldg(reinterpret_cast<const uint2*>(row + l * 8));
    else
      w[0] = __ldg(reinterpret_cast<const uint32_t*>(row + l * 4));
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int c = static_cast<int>((w[i * BITS / 32] >> (i * BITS % 32)) & ((1u << BITS) - 1u));
      out[i] = kc16<T>(s * static_cast<float>(c - z));
    }
  }
  *reinterpret_cast<uint4*>(static_cast<T*>(isv ? p.vo : p.ko) + (t * p.heads + h) * D + l * 8) =
      *reinterpret_cast<const uint4*>(out);
}

template <typename T, int D>
void launch_cache(const CacheArgs& a, int bits, bool write, cudaStream_t s) {
  const int64_t threads = a.count * 2 * a.heads * (D / 8);
  const unsigned grid = static_cast<unsigned>((threads + KC_THREADS - 1) / KC_THREADS);
  if (write) {
    if (bits == 16)
      cache_write_kernel<T, D, 16><<<grid, KC_THREADS, 0, s>>>(a);
    else if (bits == 8)
      cache_write_kernel<T, D, 8><<<grid, KC_THREADS, 0, s>>>(a);
    else
      cache_write_kernel<T, D, 4><<<grid, KC_THREADS, 0, s>>>(a);
  } else {
    if (bits == 16)
      cache_read_kernel<T, D, 16><<<grid, KC_THREADS, 0, s>>>(a);
    else if (bits == 8)
      cache_read_kernel<T, D, 8><<<grid, KC_THREADS, 0, s>>>(a);
    else
      cache_read_kernel<T, D, 4><<<grid, KC_THREADS, 0, s>>>(a);
  }
}

int launch_cache(const CacheArgs& a, int dtype, int head_dim, int bits, bool write, cudaStream_t s) {
  if (dtype == GPTQ_BF16) {
    if (head_dim == 128)
      launch_cache<__nv_bfloat16, 128>(a, bits, write, s);
    else
      launch_cache<__nv_bfloat16, 64>(a, bits, write, s);
  } else {
    if (head_dim == 128)
      launch_cache<__half, 128>(a, bits, write, s);
    else
      launch_cache<__half, 64>(a, bits, write, s);
  }
  return after_launch();
}

}  // namespace

int check_cache(const void* kc, const void* vc, const float* ks, const uint8_t* kz, const float* vs, const uint8_t* vz,
                int bits, int64_t pages, int page_size, int kv_heads, int head_dim, int dtype) {
  if (!kc || !vc || pages <= 0 || page_size <= 0 || kv_heads <= 0 || head_dim <= 0) return GPTQ_ERR_INVALID_ARG;
  if (dtype != GPTQ_F16 && dtype != GPTQ_BF16) return GPTQ_ERR_INVALID_ARG;
  if (bits != 16 && bits != 8 && bits != 4) return GPTQ_ERR_INVALID_ARG;
  if (bits < 16 && (!ks || !kz || !vs || !vz)) return GPTQ_ERR_INVALID_ARG;
  if (head_dim != 64 && head_dim != 128) return GPTQ_ERR_UNSUPPORTED;
  if (page_size < 16 || page_size > 256 || (page_size & (page_size - 1))) return GPTQ_ERR_UNSUPPORTED;
  if (kv_heads > 4096 || pages * page_size > 2147483647LL) return GPTQ_ERR_UNSUPPORTED;  // slots are 32-bit
  if (!aligned16(kc) || !aligned16(vc)) return GPTQ_ERR_UNSUPPORTED;
  if (bits < 16 && (!aligned16(ks) || !aligned16(kz) || !aligned16(vs) || !aligned16(vz))) return GPTQ_ERR_UNSUPPORTED;
  return GPTQ_OK;
}

}  // namespace gptq

using namespace gptq;

extern "C" int gptq_cache_write(const void* k, const void* v, int dtype, int64_t tokens, int kv_heads, int head_dim,
                                int64_t k_token_stride, int64_t k_head_stride, int64_t v_token_stride,
                                int64_t v_head_stride, void* k_cache, void* v_cache, float* k_scales,
                                uint8_t* k_zeros, float* v_scales, uint8_t* v_zeros, int bits, int64_t pages,
                                int page_size, const int32_t* slots, void* stream) {
  if (tokens < 0 || (tokens > 0 && (!k || !v || !slots))) return GPTQ_ERR_INVALID_ARG;
  GPTQ_TRY(check_cache(k_cache, v_cache, k_scales, k_zeros, v_scales, v_zeros, bits, pages, page_size, kv_heads,
                       head_dim, dtype));
  if (((k_token_stride | k_head_stride | v_token_stride | v_head_stride) & 7) || !aligned16(k) || !aligned16(v))
    return GPTQ_ERR_UNSUPPORTED;
  if (tokens * 2 * kv_heads * (head_dim / 8) / KC_THREADS >= 2147483647LL) return GPTQ_ERR_UNSUPPORTED;
  if (tokens == 0) return GPTQ_OK;
  int shift = 0;
  while ((1 << shift) < page_size) ++shift;
  CacheArgs a{k, v, nullptr, nullptr, k_token_stride, k_head_stride, v_token_stride, v_head_stride, k_cache, v_cache,
              k_scales, v_scales, k_zeros, v_zeros, tokens, pages * page_size, kv_heads, shift, slots};
  return launch_cache(a, dtype, head_dim, bits, true, static_cast<cudaStream_t>(stream));
}

extern "C" int gptq_cache_read(const void* k_cache, const void* v_cache, const float* k_scales,
                               const uint8_t* k_zeros, const float* v_scales, const uint8_t* v_zeros, int bits,
                               int64_t pages, int page_size, const int32_t* slots, int64_t count, int kv_heads,
                               int head_dim, int dtype, void* k, void* v, void* stream) {
  if (count < 0 || (count > 0 && (!k || !v || !slots))) return GPTQ_ERR_INVALID_ARG;
  GPTQ_TRY(check_cache(k_cache, v_cache, k_scales, k_zeros, v_scales, v_zeros, bits, pages, page_size, kv_heads,
                       head_dim, dtype));
  if (!aligned16(k) || !aligned16(v)) return GPTQ_ERR_UNSUPPORTED;
  if (count * 2 * kv_heads * (head_dim / 8) / KC_THREADS >= 2147483647LL) return GPTQ_ERR_UNSUPPORTED;
  if (count == 0) return GPTQ_OK;
  int shift = 0;
  while ((1 << shift) < page_size) ++shift;
  CacheArgs a{nullptr, nullptr, k, v, 0, 0, 0, 0, const_cast<void*>(k_cache), const_cast<void*>(v_cache),
              const_cast<float*>(k_scales), const_cast<float*>(v_scales), const_cast<uint8_t*>(k_zeros),
              const_cast<uint8_t*>(v_zeros), count, pages * page_size, kv_heads, shift, slots};
  return launch_cache(a, dtype, head_dim, bits, false, static_cast<cudaStream_t>(stream));
}
