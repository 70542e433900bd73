// A paged key/value cache: quantizing vectors as they are written, and reading them back.
//
// One vector (a token's key or value of one kv head, D = 64 or 128 values) is one group of the
// library's uniform quantizer: scale = (hi - lo) / maxq over a range that holds 0, an integer
// zero point, value = scale * (code - zero).  The code is the one nearest to the exact quotient
// x / s (half to even): k = rint(x * (1/s)) is at most one off, and only where x * (1/s) lies
// within its error of a half; there the remainder x - k s, which one fused multiply-add gives
// exactly, settles it against s / 2.  So the codes do not depend on how a division rounds.
//
// Both directions are bound by memory as long as a value costs few instructions: rounding by
// adding 1.5 2^23 (the code is then the low byte), the range by packed 16-bit maxima of (x, -x)
// that carry NaN along, the exact step behind a test of all 8 values.  (With the exact step for
// every value and 64-bit index divisions, 8192 tokens of 32 heads of 128 took 80 us to write in 4 bits and
// 80 to read; now 64 and 38, where the bytes take 26 each, and 43 and 44 in 16 bits, 6.1 TB/s.)  A vector is D/8 neighbouring threads with 8 values (16 bytes) each: its range is a
// shuffle over them, and the codes leave as 8 or 4 bytes per thread.  Keys and values go in one launch.
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
  uint32_t per, magic;  // vectors of a token (keys and values of all heads), 2^32 / per rounded down
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

constexpr float ROUND = 12582912.f;  // 1.5 2^23: adding it rounds to an integer, in the low bits of the sum

// Largest of pairs, NaN where one is NaN.
template <typename T>
__device__ __forceinline__ uint32_t max_pair(uint32_t a, uint32_t b);
template <>
__device__ __forceinline__ uint32_t max_pair<__nv_bfloat16>(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
template <>
__device__ __forceinline__ uint32_t max_pair<__half>(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

// Token (or slot) of a vector, and its side and head.
__device__ __forceinline__ uint32_t token_of(const CacheArgs& p, uint32_t vec, int& sh) {
  uint32_t t = __umulhi(vec, p.magic), rem = vec - t * p.per;
  if (rem >= p.per) {
    ++t;
    rem -= p.per;
  }
  sh = static_cast<int>(rem);
  return t;
}

// Offset (in vectors) of slot s, head h in [pages, heads, page_size]; -1 outside the cache.
__device__ __forceinline__ int64_t vector_at(const CacheArgs& p, int slot, int h) {
  if (slot < 0 || slot >= p.slots_total) return -1;
  const int64_t page = slot >> p.page_shift;
  return ((page * p.heads + h) << p.page_shift) + (slot & ((1 << p.page_shift) - 1));
}

// Packed fp32 pairs (the f32x2 arithmetic of sm_100).
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;"
      : "=l"(reinterpret_cast<unsigned long long&>(d))
      : "l"(reinterpret_cast<unsigned long long&>(a)), "l"(reinterpret_cast<unsigned long long&>(b)),
        "l"(reinterpret_cast<unsigned long long&>(c)));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("add.rn.f32x2 %0, %1, %2;"
      : "=l"(reinterpret_cast<unsigned long long&>(d))
      : "l"(reinterpret_cast<unsigned long long&>(a)), "l"(reinterpret_cast<unsigned long long&>(b)));
  return d;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 d;
  asm("mul.rn.f32x2 %0, %1, %2;"
      : "=l"(reinterpret_cast<unsigned long long&>(d))
      : "l"(reinterpret_cast<unsigned long long&>(a)), "l"(reinterpret_cast<unsigned long long&>(b)));
  return d;
}
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }

// The 8 values of a thread as pairs.
__device__ __forceinline__ void widen(const uint4 raw, float2 (&x)[4], __nv_bfloat16) {
  const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) x[i] = make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
}
__device__ __forceinline__ void widen(const uint4 raw, float2 (&x)[4], __half) {
  const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) x[i] = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
}

// Bytes added without carries between them.
__device__ __forceinline__ uint32_t add_bytes(uint32_t a, uint32_t b) {
  return ((a & 0x7f7f7f7fu) + (b & 0x7f7f7f7fu)) ^ ((a ^ b) & 0x80808080u);
}

// (largest, largest of the negatives) of a thread's values and 0, NaN where one is NaN.
template <typename T>
__device__ __forceinline__ uint32_t ends_of(const uint4 raw) {
  constexpr uint32_t FLIP = 0x80008000u;
  const uint32_t top = max_pair<T>(max_pair<T>(raw.x, raw.y), max_pair<T>(raw.z, raw.w));
  const uint32_t low = max_pair<T>(max_pair<T>(raw.x ^ FLIP, raw.y ^ FLIP), max_pair<T>(raw.z ^ FLIP, raw.w ^ FLIP));
  return max_pair<T>(max_pair<T>(__byte_perm(top, low, 0x5410u), __byte_perm(top, low, 0x7632u)), 0u);
}

// Scale, its reciprocal and the zero point of a vector from its ends.  A vector with a NaN, an infinity or a range
// over float32's: scale NaN.
struct Params {
  float s, inv, z;
};
template <typename T, int BITS>
__device__ __forceinline__ Params params_of(uint32_t ends) {
  constexpr float MAXQ = static_cast<float>((1 << BITS) - 1);
  float hi = to_f32(reinterpret_cast<const T*>(&ends)[0]), lo = -to_f32(reinterpret_cast<const T*>(&ends)[1]);
  if (lo == 0.f && hi == 0.f) {
    lo = -1.f;
    hi = 1.f;
  }
  Params p;
  p.s = __fdiv_rn(hi - lo, MAXQ);
  p.inv = 0.f;
  p.z = 0.f;
  if (p.s < INFINITY) {
    const float up = p.s < 0x1p-100f ? 0x1p64f : 1.f;  // as in store_vector
    p.inv = __fdiv_rn(1.f, p.s * up);
    p.z = fminf(fmaxf(rint_quotient(-lo * up, p.s * up, p.inv), 0.f), MAXQ);
  } else {
    p.s = __int_as_float(0x7fc00000);
  }
  return p;
}

// One vector's codes, scale and zero point, stored at vector `at` (at < 0: none).
template <typename T, int D, int BITS>
__device__ __forceinline__ void store_vector(const CacheArgs& p, bool isv, int64_t at, int l, const uint4 raw,
                                             const Params q) {
  if (at < 0) return;
  uint8_t* row = static_cast<uint8_t*>(isv ? p.vc : p.kc) + at * (D * BITS / 8);
  if constexpr (BITS == 16) {
    *reinterpret_cast<uint4*>(row + l * 16) = raw;
  } else {
    constexpr float MAXQ = static_cast<float>((1 << BITS) - 1);
    uint32_t c[2] = {0, 0};  // codes as bytes
    if (q.s == q.s) {
      // tiny scales are brought up by a power of two (exactly), where 1/s is finite
      const float up = q.s < 0x1p-100f ? 0x1p64f : 1.f;
      const float su = q.s * up;
      float2 x[4], t[4];
      widen(raw, x, T());
      float far = 0.f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x[i] = mul2(x[i], both(up));
        t[i] = fma2(x[i], both(q.inv), both(ROUND));
        const float2 k = add2(t[i], both(-ROUND));
        const float2 e = fma2(k, both(-su), x[i]);  // exact, as in rint_quotient
        far = fmaxf(far, fmaxf(fabsf(e.x), fabsf(e.y)));
      }
      if (!(far < 0.5f * su)) {  // a tie, or one off beside a half
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          t[i].x = rint_quotient(x[i].x, su, q.inv) + ROUND;
          t[i].y = rint_quotient(x[i].y, su, q.inv) + ROUND;
        }
      }
      // x >= lo leaves code >= 0 (rounding is odd); hi and zero may both round up
      const float lim = ROUND + (MAXQ - q.z);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint32_t lo = __byte_perm(__float_as_uint(fminf(t[2 * i].x, lim)), __float_as_uint(fminf(t[2 * i].y, lim)), 0x0040u);
        const uint32_t hi =
            __byte_perm(__float_as_uint(fminf(t[2 * i + 1].x, lim)), __float_as_uint(fminf(t[2 * i + 1].y, lim)), 0x0040u);
        c[i] = add_bytes(__byte_perm(lo, hi, 0x5410u), static_cast<uint32_t>(q.z) * 0x01010101u);
      }
    }
    if constexpr (BITS == 8) {
      *reinterpret_cast<uint2*>(row + l * 8) = make_uint2(c[0], c[1]);
    } else {
      // two codes to a byte
      *reinterpret_cast<uint32_t*>(row + l * 4) = __byte_perm(c[0] | (c[0] >> 4), c[1] | (c[1] >> 4), 0x6420u);
    }
    if (l == 0) {
      (isv ? p.vs : p.ks)[at] = q.s;
      (isv ? p.vz : p.kz)[at] = static_cast<uint8_t>(q.z);
    }
  }
}

// U tokens per thread, of one side and head, so that addresses cost one addition each; loads before anything
// that waits for them: a thread's two loads depend on one another (slot, then vector).  Few vectors: one per
// thread, for the shortest way through.
template <typename T, int D, int BITS, int U>
__global__ void __launch_bounds__(KC_THREADS) cache_write_kernel(const CacheArgs p) {
  constexpr int LPV = D / 8;             // threads of a vector
  constexpr int VPC = KC_THREADS / LPV;  // vectors of a CTA at a time
  const int l = threadIdx.x % LPV;
  int64_t at[U];
  uint4 raw[U];
  // (tokens, side, head): the LPV threads of a vector never cross a warp
  int sh;
  const int64_t t = static_cast<int64_t>(token_of(p, blockIdx.x * VPC + threadIdx.x / LPV, sh)) * U;
  const bool isv = sh >= p.heads;
  const int h = isv ? sh - p.heads : sh;
  const int64_t step = isv ? p.v_ts : p.k_ts;
  const T* src = static_cast<const T*>(isv ? p.v : p.k) + t * step + h * (isv ? p.v_hs : p.k_hs) + l * 8;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    raw[u] = make_uint4(0, 0, 0, 0);
    at[u] = -1;
    if (t + u < p.count) {
      at[u] = __ldg(p.slots + t + u);
      raw[u] = __ldg(reinterpret_cast<const uint4*>(src + u * step));
    }
  }
#pragma unroll
  for (int u = 0; u < U; ++u) at[u] = vector_at(p, static_cast<int>(at[u]), h);
  Params q[U];
  if constexpr (BITS < 16) {
    uint32_t mine = 0;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      uint32_t ends = ends_of<T>(raw[u]);
#pragma unroll
      for (int o = LPV / 2; o; o >>= 1) ends = max_pair<T>(ends, __shfl_xor_sync(0xffffffffu, ends, o));
      if (l % U == u) mine = ends;
    }
    // the vectors' divisions, each by another lane of its threads
    const Params own = params_of<T, BITS>(mine);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      q[u].s = __shfl_sync(0xffffffffu, own.s, u, LPV);
      q[u].inv = __shfl_sync(0xffffffffu, own.inv, u, LPV);
      q[u].z = __shfl_sync(0xffffffffu, own.z, u, LPV);
    }
  }
#pragma unroll
  for (int u = 0; u < U; ++u) store_vector<T, D, BITS>(p, isv, at[u], l, raw[u], q[u]);
}

template <typename T, int D, int BITS, int U>
__global__ void __launch_bounds__(KC_THREADS) cache_read_kernel(const CacheArgs p) {
  constexpr int LPV = D / 8;
  constexpr int VPC = KC_THREADS / LPV;
  constexpr int W = BITS / 4;  // words of a thread's 8 values
  const int l = threadIdx.x % LPV;
  int64_t at[U];
  int sh;
  const int64_t t = static_cast<int64_t>(token_of(p, blockIdx.x * VPC + threadIdx.x / LPV, sh)) * U;
  const bool isv = sh >= p.heads;
  const int h = isv ? sh - p.heads : sh;
  T* dst = static_cast<T*>(isv ? p.vo : p.ko) + (t * p.heads + h) * D + l * 8;
  const int step = p.heads * D;
#pragma unroll
  for (int u = 0; u < U; ++u) at[u] = t + u < p.count ? __ldg(p.slots + t + u) : -1;
#pragma unroll
  for (int u = 0; u < U; ++u) at[u] = vector_at(p, static_cast<int>(at[u]), h);
  uint32_t w[U][W];
  float scale[U], zero[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
#pragma unroll
    for (int i = 0; i < W; ++i) w[u][i] = 0;
    scale[u] = 0.f;  // outside the cache: zeros
    zero[u] = 8388608.f;
    if (at[u] < 0) continue;
    const uint8_t* from = static_cast<const uint8_t*>(isv ? p.vc : p.kc) + at[u] * (D * BITS / 8) + l * BITS;
    if constexpr (W == 4) {
      *reinterpret_cast<uint4*>(w[u]) = __ldg(reinterpret_cast<const uint4*>(from));
    } else {
      if constexpr (W == 2)
        *reinterpret_cast<uint2*>(w[u]) = __ldg(reinterpret_cast<const uint2*>(from));
      else
        w[u][0] = __ldg(reinterpret_cast<const uint32_t*>(from));
      scale[u] = __ldg((isv ? p.vs : p.ks) + at[u]);
      zero[u] = __uint_as_float(0x4B000000u | __ldg((isv ? p.vz : p.kz) + at[u]));  // 2^23 + zero
    }
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    if (t + u >= p.count) break;
    alignas(16) T out[8];
    if constexpr (BITS == 16) {
      *reinterpret_cast<uint4*>(out) = *reinterpret_cast<const uint4*>(w[u]);
    } else {
#pragma unroll
      for (int i = 0; i < 8; i += 2) {
        const uint32_t v = w[u][i * BITS / 32] >> (i * BITS % 32);
        float2 f;  // 2^23 + code
        if constexpr (BITS == 8) {
          f.x = __uint_as_float(__byte_perm(v, 0x4B000000u, 0x7650u));
          f.y = __uint_as_float(__byte_perm(v, 0x4B000000u, 0x7651u));
        } else {
          f.x = __uint_as_float((v & 15u) | 0x4B000000u);
          f.y = __uint_as_float(((v >> 4) & 15u) | 0x4B000000u);
        }
        f = mul2(both(scale[u]), add2(f, both(-zero[u])));  // the difference is exact
        out[i] = kc16<T>(f.x);
        out[i + 1] = kc16<T>(f.y);
      }
    }
    *reinterpret_cast<uint4*>(dst + u * step) = *reinterpret_cast<const uint4*>(out);
  }
}

template <typename T, int D, int U>
void launch_cache(const CacheArgs& a, int bits, bool write, cudaStream_t s) {
  constexpr int VPC = KC_THREADS / (D / 8);
  const unsigned grid = static_cast<unsigned>(((a.count + U - 1) / U * 2 * a.heads + VPC - 1) / VPC);
  if (write) {
    if (bits == 16)
      cache_write_kernel<T, D, 16, U><<<grid, KC_THREADS, 0, s>>>(a);
    else if (bits == 8)
      cache_write_kernel<T, D, 8, U><<<grid, KC_THREADS, 0, s>>>(a);
    else
      cache_write_kernel<T, D, 4, U><<<grid, KC_THREADS, 0, s>>>(a);
  } else {
    if (bits == 16)
      cache_read_kernel<T, D, 16, U><<<grid, KC_THREADS, 0, s>>>(a);
    else if (bits == 8)
      cache_read_kernel<T, D, 8, U><<<grid, KC_THREADS, 0, s>>>(a);
    else
      cache_read_kernel<T, D, 4, U><<<grid, KC_THREADS, 0, s>>>(a);
  }
}

template <typename T, int D>
void launch_cache(const CacheArgs& a, int bits, bool write, cudaStream_t s) {
  if (a.count * 2 * a.heads >= 16384)
    launch_cache<T, D, 4>(a, bits, write, s);
  else
    launch_cache<T, D, 1>(a, bits, write, s);
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
  if (tokens * 2 * kv_heads > (int64_t(1) << 31)) return GPTQ_ERR_UNSUPPORTED;
  if (tokens == 0) return GPTQ_OK;
  int shift = 0;
  while ((1 << shift) < page_size) ++shift;
  CacheArgs a{k, v, nullptr, nullptr, k_token_stride, k_head_stride, v_token_stride, v_head_stride, k_cache, v_cache,
              k_scales, v_scales, k_zeros, v_zeros, tokens, pages * page_size, kv_heads, shift, 2u * kv_heads,
              static_cast<uint32_t>((uint64_t(1) << 32) / (2u * kv_heads)), slots};
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
  if (count * 2 * kv_heads > (int64_t(1) << 31)) return GPTQ_ERR_UNSUPPORTED;
  if (count == 0) return GPTQ_OK;
  int shift = 0;
  while ((1 << shift) < page_size) ++shift;
  CacheArgs a{nullptr, nullptr, k, v, 0, 0, 0, 0, const_cast<void*>(k_cache), const_cast<void*>(v_cache),
              const_cast<float*>(k_scales), const_cast<float*>(v_scales), const_cast<uint8_t*>(k_zeros),
              const_cast<uint8_t*>(v_zeros), count, pages * page_size, kv_heads, shift, 2u * kv_heads,
              static_cast<uint32_t>((uint64_t(1) << 32) / (2u * kv_heads)), slots};
  return launch_cache(a, dtype, head_dim, bits, false, static_cast<cudaStream_t>(stream));
}
