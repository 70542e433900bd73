// Rotary positions on the queries and keys of a step's tokens, in one launch.
//
// The pairs (a, b) of the first r values of a head turn by theta = p_t f_i:
//   a' = A (a cos theta - b sin theta),  b' = A (b cos theta + a sin theta).
// theta / pi is formed and reduced modulo 2 in double precision (a position of 10^6 leaves
// 2^-33 of a turn), its sine and cosine are then taken in fp32 on the reduced angle, and the
// rotation is one fp32 pass rounded once to 16 bits.
//
// Bound by memory: each value is read and written once.  A CTA takes kTok tokens: its threads
// compute the tokens' cosines and sines once into shared memory (64 double products per token
// of 128-wide heads, shared by all heads), then walk the (token, head, 8 pairs) items, 32
// bytes each, neighbouring threads on neighbouring chunks of a head.  16384 tokens of 64 + 8
// heads of 128: 108 us and 5.6 TB/s among calls with other inputs (99 and 6.1 from a graph that replays one); 8 tokens
// of 32 + 32: 2.4 us, a launch.  Where rotary_dim is no multiple of 16, value by value: 781 us with 20 of 128 rotated.
#include <math.h>

#include <algorithm>

#include "common.cuh"

namespace gptq {
namespace {

constexpr int RT_THREADS = 256;
constexpr int RT_MAX_PAIRS = 256;  // head_dim <= 512

struct RotaryArgs {
  const void *q, *k;
  void *qo, *ko;
  int64_t tokens, q_ts, q_hs, k_ts, k_hs, qo_ts, qo_hs, ko_ts, ko_hs;
  int heads, kv_heads, d, r;
  const int32_t* pos;
  const double* freq;
  float factor;
};

template <typename T>
__device__ __forceinline__ T rt16(float v);
template <>
__device__ __forceinline__ __half rt16<__half>(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ __nv_bfloat16 rt16<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

template <typename T>
union Vec8 {
  uint4 u;
  T e[8];
};

// VEC: rotary_dim is a multiple of 16, so that 8 pairs are whole 16-byte vectors in both
// layouts; otherwise items are single pairs and single copied values.
template <typename T, bool VEC, bool INTER, int TOK>
__global__ void __launch_bounds__(RT_THREADS) rotary_kernel(const RotaryArgs p) {
  __shared__ float2 cs[TOK * RT_MAX_PAIRS];
  const int half = p.r / 2;
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * TOK;
  const int nt = static_cast<int>(min(static_cast<int64_t>(TOK), p.tokens - t0));
  for (int e = threadIdx.x; e < nt * half; e += RT_THREADS) {
    const int tt = TOK == 1 ? 0 : e / half, i = e - tt * half;
    const double turns = static_cast<double>(__ldg(p.pos + t0 + tt)) * __ldg(p.freq + i) * 0.31830988618379067154;
    const float x = static_cast<float>(turns - 2.0 * rint(turns * 0.5));  // in units of pi, |x| <= 1
    float sn, cn;
    sincospif(x, &sn, &cn);
    cs[tt * half + i] = make_float2(cn * p.factor, sn * p.factor);
  }
  __syncthreads();
  const int rot = VEC ? half / 8 : half;               // rotated items of a head
  const int copy = VEC ? (p.d - p.r) / 8 : p.d - p.r;  // copied items
  const int per = rot + copy, all = p.heads + p.kv_heads;
  const int lo = blockIdx.y * ((all + gridDim.y - 1) / gridDim.y);
  const int nh = min(all, lo + static_cast<int>((all + gridDim.y - 1) / gridDim.y)) - lo;
  for (int e = threadIdx.x; e < nt * nh * per; e += RT_THREADS) {
    const int c = e % per, th = e / per;
    const int tt = TOK == 1 ? 0 : th / nh, h = lo + (th - tt * nh);
    const bool isq = h < p.heads;
    const int hh = isq ? h : h - p.heads;
    const int64_t t = t0 + tt;
    const T* src = static_cast<const T*>(isq ? p.q : p.k) + t * (isq ? p.q_ts : p.k_ts) + hh * (isq ? p.q_hs : p.k_hs);
    T* dst = static_cast<T*>(isq ? p.qo : p.ko) + t * (isq ? p.qo_ts : p.ko_ts) + hh * (isq ? p.qo_hs : p.ko_hs);
    if (c >= rot) {
      if (src == dst) continue;
      const int o = VEC ? p.r + (c - rot) * 8 : p.r + (c - rot);
      if constexpr (VEC)
        *reinterpret_cast<uint4*>(dst + o) = *reinterpret_cast<const uint4*>(src + o);
      else
        dst[o] = src[o];
      continue;
    }
    if constexpr (VEC) {
      const int oa = INTER ? c * 16 : c * 8, ob = INTER ? c * 16 + 8 : half + c * 8;
      Vec8<T> a, b, x, y;
      a.u = *reinterpret_cast<const uint4*>(src + oa);
      b.u = *reinterpret_cast<const uint4*>(src + ob);
      const float2* w = cs + tt * half + c * 8;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float2 f = w[i];
        const float u = to_f32(INTER ? (i < 4 ? a.e[(2 * i) & 7] : b.e[(2 * i) & 7]) : a.e[i]);
        const float v = to_f32(INTER ? (i < 4 ? a.e[(2 * i + 1) & 7] : b.e[(2 * i + 1) & 7]) : b.e[i]);
        const T m = rt16<T>(u * f.x - v * f.y), n = rt16<T>(v * f.x + u * f.y);
        if constexpr (INTER) {
          (i < 4 ? x : y).e[(2 * i) & 7] = m;
          (i < 4 ? x : y).e[(2 * i + 1) & 7] = n;
        } else {
          x.e[i] = m;
          y.e[i] = n;
        }
      }
      *reinterpret_cast<uint4*>(dst + oa) = x.u;
      *reinterpret_cast<uint4*>(dst + ob) = y.u;
    } else {
      const int oa = INTER ? 2 * c : c, ob = INTER ? 2 * c + 1 : half + c;
      const float2 f = cs[tt * half + c];
      const float u = to_f32(src[oa]), v = to_f32(src[ob]);
      dst[oa] = rt16<T>(u * f.x - v * f.y);
      dst[ob] = rt16<T>(v * f.x + u * f.y);
    }
  }
}

template <typename T, bool VEC, bool INTER>
void launch_rotary(const RotaryArgs& a, cudaStream_t s) {
  // Four tokens per CTA share one round of cosines; few tokens: one per CTA, its heads over
  // as many CTAs as fill the SMs.
  const int sms = num_sms();
  if (a.tokens >= 4 * sms) {
    rotary_kernel<T, VEC, INTER, 4><<<static_cast<unsigned>((a.tokens + 3) / 4), RT_THREADS, 0, s>>>(a);
  } else {
    const int items = (a.heads + a.kv_heads) * std::max(1, a.d / 16);
    const unsigned most = static_cast<unsigned>(std::max(1, items / RT_THREADS));
    const unsigned want = static_cast<unsigned>(std::max<int64_t>(1, 2 * sms / a.tokens));
    rotary_kernel<T, VEC, INTER, 1><<<dim3(static_cast<unsigned>(a.tokens), std::min(most, want)), RT_THREADS, 0, s>>>(a);
  }
}

template <typename T>
void launch_rotary(const RotaryArgs& a, bool inter, cudaStream_t s) {
  const bool vec = a.r % 16 == 0;
  if (vec && inter)
    launch_rotary<T, true, true>(a, s);
  else if (vec)
    launch_rotary<T, true, false>(a, s);
  else if (inter)
    launch_rotary<T, false, true>(a, s);
  else
    launch_rotary<T, false, false>(a, s);
}

}  // namespace
}  // namespace gptq

using namespace gptq;

extern "C" int gptq_rotary_frequencies(int rotary_dim, double base, int scaling, double factor, int64_t original_len,
                                       double beta_fast, double beta_slow, double* inv_freq,
                                       float* attention_factor) {
  const int r = rotary_dim;
  if (!inv_freq || !attention_factor || r <= 0 || r % 2 || !(base > 1.0) || !std::isfinite(base))
    return GPTQ_ERR_INVALID_ARG;
  if (scaling < GPTQ_ROTARY_NONE || scaling > GPTQ_ROTARY_YARN) return GPTQ_ERR_INVALID_ARG;
  if (scaling != GPTQ_ROTARY_NONE && !(factor >= 1.0 && std::isfinite(factor))) return GPTQ_ERR_INVALID_ARG;
  if (scaling == GPTQ_ROTARY_NTK && r <= 2) return GPTQ_ERR_INVALID_ARG;
  if (scaling == GPTQ_ROTARY_YARN &&
      !(original_len > 0 && beta_slow > 0.0 && beta_fast > beta_slow && std::isfinite(beta_fast)))
    return GPTQ_ERR_INVALID_ARG;
  if (scaling == GPTQ_ROTARY_NTK) base *= pow(factor, static_cast<double>(r) / (r - 2));
  *attention_factor = 1.f;
  double lo = 0, hi = 0;
  if (scaling == GPTQ_ROTARY_YARN) {
    // the (fractional) pair that turns beta times in the original length: base^(2i/r) = L / (2 pi beta)
    auto at = [&](double beta) {
      return r * log(static_cast<double>(original_len) / (2.0 * M_PI * beta)) / (2.0 * log(base));
    };
    lo = std::max(floor(at(beta_fast)), 0.0);
    hi = std::min(ceil(at(beta_slow)), static_cast<double>(r - 1));
    *attention_factor = factor > 1.0 ? static_cast<float>(0.1 * log(factor) + 1.0) : 1.f;
  }
  for (int i = 0; i < r / 2; ++i) {
    double f = pow(base, -2.0 * i / r);
    if (scaling == GPTQ_ROTARY_LINEAR) f /= factor;
    if (scaling == GPTQ_ROTARY_YARN) {
      const double keep = 1.0 - std::min(std::max((i - lo) / std::max(hi - lo, 1e-3), 0.0), 1.0);
      f = f / factor * (1.0 - keep) + f * keep;
    }
    inv_freq[i] = f;
  }
  return GPTQ_OK;
}

extern "C" int gptq_rotary(const void* q, const void* k, int dtype, int64_t tokens, int heads, int kv_heads,
                           int head_dim, int rotary_dim, int interleaved, int64_t q_token_stride,
                           int64_t q_head_stride, int64_t k_token_stride, int64_t k_head_stride,
                           const int32_t* positions, const double* inv_freq, float attention_factor, void* q_out,
                           void* k_out, int64_t qo_token_stride, int64_t qo_head_stride, int64_t ko_token_stride,
                           int64_t ko_head_stride, void* stream) {
  if (!inv_freq || tokens < 0 || heads <= 0 || kv_heads < 0) return GPTQ_ERR_INVALID_ARG;
  if (tokens > 0 && (!q || !q_out || !positions || (kv_heads > 0 && (!k || !k_out)))) return GPTQ_ERR_INVALID_ARG;
  if (dtype != GPTQ_F16 && dtype != GPTQ_BF16) return GPTQ_ERR_INVALID_ARG;
  if (head_dim <= 0 || rotary_dim <= 0 || rotary_dim % 2 || rotary_dim > head_dim) return GPTQ_ERR_INVALID_ARG;
  if (head_dim % 8 || head_dim > 2 * RT_MAX_PAIRS || heads > 65535 || kv_heads > 65535 || tokens > (int64_t(1) << 30))
    return GPTQ_ERR_UNSUPPORTED;
  const bool hk = kv_heads > 0;
  if (((q_token_stride | q_head_stride | qo_token_stride | qo_head_stride) & 7) || !aligned16(q) || !aligned16(q_out) ||
      (hk && (((k_token_stride | k_head_stride | ko_token_stride | ko_head_stride) & 7) || !aligned16(k) ||
              !aligned16(k_out))))
    return GPTQ_ERR_UNSUPPORTED;
  // in place only where every value keeps its address
  if ((tokens > 0 && q == q_out && (q_token_stride != qo_token_stride || q_head_stride != qo_head_stride)) ||
      (tokens > 0 && hk && k == k_out && (k_token_stride != ko_token_stride || k_head_stride != ko_head_stride)))
    return GPTQ_ERR_INVALID_ARG;
  if (tokens == 0) return GPTQ_OK;
  RotaryArgs a{q,  k,  q_out, k_out, tokens, q_token_stride, q_head_stride, k_token_stride, k_head_stride,
               qo_token_stride, qo_head_stride, ko_token_stride, ko_head_stride, heads, kv_heads, head_dim, rotary_dim,
               positions, inv_freq, attention_factor};
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (dtype == GPTQ_BF16)
    launch_rotary<__nv_bfloat16>(a, interleaved != 0, s);
  else
    launch_rotary<__half>(a, interleaved != 0, s);
  return after_launch();
}
