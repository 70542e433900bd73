// Attention over a paged cache for sequences with few rows (at most 16 rows times heads of a kv
// head: single tokens, short guesses).
//
// Each key and value byte is used for at most 16 rows, so the cache's bytes bound the kernel and
// everything serves keeping loads in flight:
//  * The rows of all query heads that share a kv head are one 16-row tile (row i * group + g), so a
//    cache line is read once.  Scores and the weighted sum run on the 16x8x16 matrix instruction.
//  * Keys and values go from global memory to registers in the layout of that instruction's operands,
//    without shared memory: the order of the contraction index is free as long as both operands agree,
//    so a lane takes contiguous 16-byte pieces of a key and the query is laid out to match; for the
//    values the column order is free, and a lane takes contiguous pieces of four keys.
//  * Codes enter the products as the integers code - zero (exact in both 16-bit types, at most 255);
//    a key's scale multiplies its scores afterwards, a value's scale its probability, so
//    dequantizing costs one or two instructions per pair of codes and no rounding of its own.  The
//    scaled probabilities are rounded to bfloat16, whose range holds any scale.
//  * The keys of all sequences are one line of 64-key units, cut into equal shares, one per resident
//    CTA: ragged lengths balance, and one long sequence fills the GPU.  A CTA's share has at most two
//    unfinished (sequence, head) pieces, its first and its last; those leave (maximum, sum, weighted
//    sum) behind and a second launch joins them in order, so results do not depend on timing.
// Each warp walks its own keys with its own running maximum and sum (fp32); the next keys are in
// flight during the softmax, the next values during the next scores.
#include <algorithm>
#include <type_traits>

#include "paged.cuh"
#include "paged_plan.cuh"

namespace gptq {
namespace paged {
namespace {

constexpr int ST_THREADS = 128;  // 4 warps
constexpr int ST_UNIT = 64;      // keys of a unit of the line

// Words (32 bits) of a lane: of one key (a quarter of it) and of one value (an eighth).
template <int D, int BITS>
struct Lay {
  static constexpr int KW = D / 4 * BITS / 32;
  static constexpr int VW = D / 8 * BITS / 32;
  static constexpr int ROW = D * BITS / 8;                 // bytes of a vector
  static constexpr int KPW = BITS == 16 ? 16 : 32;         // keys of a warp's step
  static constexpr int NT = KPW / 8;                       // 8-key tiles of a step
  static constexpr int KP = KW >= 4 ? 4 : KW;              // words of a contiguous piece
  static constexpr int VP = VW >= 4 ? 4 : VW;
};

template <int N>
__device__ __forceinline__ void load_words(const uint8_t* p, uint32_t* w) {
  if constexpr (N == 4) {
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                 : "l"(p));
  } else if constexpr (N == 2) {
    asm volatile("ld.global.nc.L1::no_allocate.v2.u32 {%0,%1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "l"(p));
  } else {
    asm volatile("ld.global.nc.L1::no_allocate.u32 %0, [%1];" : "=r"(w[0]) : "l"(p));
  }
}

// The first of the 8 elements of a head that lane t (of 4) holds for contraction steps 2 kk, 2 kk + 1.
template <int D, int BITS>
__device__ __forceinline__ int key_elem(int t, int kk) {
  if constexpr (BITS == 16) return kk * 32 + t * 8;
  if constexpr (BITS == 8) return (kk >> 1) * 64 + t * 16 + (kk & 1) * 8;
  return t * (D / 4) + kk * 8;
}
// The element that column c (of 8) of output tile i stands for.
template <int D, int BITS>
__device__ __forceinline__ int value_elem(int c, int i) {
  if constexpr (BITS == 16) return (i >> 3) * 64 + c * 8 + (i & 7);
  return c * (D / 8) + i;
}

template <typename T>
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1);
template <>
__device__ __forceinline__ void mma<__nv_bfloat16>(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
template <>
__device__ __forceinline__ void mma<__half>(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

template <typename T>
__device__ __forceinline__ uint32_t pack2(float lo, float hi);
template <>
__device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
template <>
__device__ __forceinline__ uint32_t pack2<__half>(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// code - zero of two codes as a pair of 16-bit values, exactly.  4 bits: 0x4300 | c is the bfloat16
// 128 + c, 0x6400 | c the half 1024 + c, and bias holds 128 + zero (1024 + zero).  8 bits: 0x4B000000
// | c is the float 2^23 + c, zf holds 2^23 + zero, the difference is exact and so is its 16-bit form.
template <typename T>
__device__ __forceinline__ uint32_t sub_pair4(uint32_t nibs, uint32_t bias);
template <>
__device__ __forceinline__ uint32_t sub_pair4<__nv_bfloat16>(uint32_t nibs, uint32_t bias) {
  const uint32_t x = (nibs & 0x000f000fu) | 0x43004300u;
  const __nv_bfloat162 d = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&x),
                                   *reinterpret_cast<const __nv_bfloat162*>(&bias));
  return *reinterpret_cast<const uint32_t*>(&d);
}
template <>
__device__ __forceinline__ uint32_t sub_pair4<__half>(uint32_t nibs, uint32_t bias) {
  const uint32_t x = (nibs & 0x000f000fu) | 0x64006400u;
  const __half2 d = __hsub2(*reinterpret_cast<const __half2*>(&x), *reinterpret_cast<const __half2*>(&bias));
  return *reinterpret_cast<const uint32_t*>(&d);
}
template <typename T>
__device__ __forceinline__ uint32_t bias4(int z0, int z1) {
  if constexpr (std::is_same<T, __half>::value)
    return (0x6400u + z0) | ((0x6400u + z1) << 16);
  else
    return (0x4300u + z0) | ((0x4300u + z1) << 16);
}
template <typename T>
__device__ __forceinline__ uint32_t sub_pair8(uint32_t w0, uint32_t w1, int b0, int b1, float zf0, float zf1) {
  const float x = __uint_as_float(__byte_perm(w0, 0x4B000000u, 0x7650u + b0)) - zf0;
  const float y = __uint_as_float(__byte_perm(w1, 0x4B000000u, 0x7650u + b1)) - zf1;
  return pack2<T>(x, y);
}

template <typename T, int D, int BITS>
__global__ void __launch_bounds__(ST_THREADS, 2) step_kernel(const Args a, const Share sh, float* __restrict__ part, Cut* __restrict__ cut) {
  using Y = Lay<D, BITS>;
  using PT = typename std::conditional<BITS == 16, T, __nv_bfloat16>::type;  // type of P and V in their product
  constexpr int NT = Y::NT, NO = D / 8;
  extern __shared__ __align__(16) float red[];  // [4 warps][16][D] weighted sums, then maxima and sums
  float* red_m = red + 4 * 16 * D;
  float* red_l = red_m + 4 * 16;
  __shared__ Cursor cur_s;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  next_may_start();

  Cursor cur;
  const bool any = first_piece<ST_THREADS>(a, sh, ST_UNIT, cur, &cur_s);
  if (cut && threadIdx.x == 0)
    cut[blockIdx.x] = any ? cut_at(cur.at, cur.per, cur.u0, cur.units, sequence(a, cur.s), cur.head, 0) : Cut{0, -1};
  if (!any) return;
  const int64_t first = cur.at;
  for (; cur.at < cur.end; next_piece(a, sh, ST_UNIT, cur)) {
    const Seq q = sequence(a, cur.s);
    const int rows = q.n * a.group;
    const int h = cur.head, s = cur.s;
    const int k0 = cur.u0 * ST_UNIT, k1 = min(cur.u1 * ST_UNIT, q.len);
    const T* qbase = static_cast<const T*>(a.q);
    // keys seen by this lane's two rows
    int see[2];
    uint32_t qf[D / 16][4];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int row = g + 8 * r;
      const bool in = row < rows;
      const int i = in ? row / a.group : 0;
      see[r] = in ? min(k1, seen(a, q, i)) : 0;
      const T* qr = qbase + (q.start + i) * a.q_ts + (h * a.group + (in ? row - i * a.group : 0)) * a.q_hs;
#pragma unroll
      for (int kk = 0; kk < D / 32; ++kk) {  // 8 elements: two contraction steps
        uint4 w = make_uint4(0, 0, 0, 0);
        if (in) w = __ldg(reinterpret_cast<const uint4*>(qr + key_elem<D, BITS>(t, kk)));
        if constexpr (BITS == 4) {  // pairs (e, e + 4), as the codes' nibbles come out
          qf[2 * kk][r] = __byte_perm(w.x, w.z, 0x5410);
          qf[2 * kk][r + 2] = __byte_perm(w.x, w.z, 0x7632);
          qf[2 * kk + 1][r] = __byte_perm(w.y, w.w, 0x5410);
          qf[2 * kk + 1][r + 2] = __byte_perm(w.y, w.w, 0x7632);
        } else {
          qf[2 * kk][r] = w.x;
          qf[2 * kk][r + 2] = w.y;
          qf[2 * kk + 1][r] = w.z;
          qf[2 * kk + 1][r + 2] = w.w;
        }
      }
    }
    float o[NO][4];
#pragma unroll
    for (int i = 0; i < NO; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[i][e] = 0.f;
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};

    uint32_t kw[NT][Y::KW], vw[NT][2][Y::VW];
    int64_t vec[NT / 2], vecn[NT / 2];  // first vector of each 16 keys of the step, and of the next step
    auto find = [&](int k, int64_t (&v)[NT / 2]) {
#pragma unroll
      for (int j = 0; j < NT / 2; ++j) v[j] = k + 16 * j < k1 ? key_at(a, s, h, k + 16 * j) : 0;
    };
    // the codes' side data: zero of this lane's key per tile (keys); scales and zeros of keys 2t, 2t + 1
    int kz[NT];
    float2 ksc[NT], vsc[NT];
    int vz[NT];
    auto load_k = [&](int k, const int64_t (&v)[NT / 2]) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        if (k + (nt / 2) * 16 >= k1) continue;  // beyond the piece: scores are masked
        const int64_t at = v[nt / 2] + (nt & 1) * 8;
        const uint8_t* p = static_cast<const uint8_t*>(a.kc) + (at + g) * Y::ROW + t * Y::KP * 4;
#pragma unroll
        for (int j = 0; j < Y::KW / Y::KP; ++j) load_words<Y::KP>(p + j * 16 * Y::KP, &kw[nt][j * Y::KP]);
        if constexpr (BITS < 16) {
          kz[nt] = __ldg(a.kz + at + g);
          ksc[nt] = __ldg(reinterpret_cast<const float2*>(a.ks + at + 2 * t));
        }
      }
    };
    auto load_v = [&](int k, const int64_t (&v)[NT / 2]) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        if (k + (nt / 2) * 16 >= k1) {
#pragma unroll
          for (int e = 0; e < Y::VW; ++e) vw[nt][0][e] = vw[nt][1][e] = 0;
          if constexpr (BITS < 16) vz[nt] = 0;
          continue;
        }
        const int64_t at = v[nt / 2] + (nt & 1) * 8 + 2 * t;
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const uint8_t* p = static_cast<const uint8_t*>(a.vc) + (at + r) * Y::ROW + g * Y::VP * 4;
#pragma unroll
          for (int j = 0; j < Y::VW / Y::VP; ++j) load_words<Y::VP>(p + j * 32 * Y::VP, &vw[nt][r][j * Y::VP]);
        }
        if constexpr (BITS < 16) {
          vz[nt] = __ldg(reinterpret_cast<const uint16_t*>(a.vz + at));
          vsc[nt] = __ldg(reinterpret_cast<const float2*>(a.vs + at));
        }
      }
    };

    int k = k0 + warp * Y::KPW;
    constexpr int STRIDE = 4 * Y::KPW;
    if (k < k1) {
      find(k, vec);
      load_k(k, vec);
      load_v(k, vec);
      find(k + STRIDE, vecn);
    }
    for (; k < k1; k += STRIDE) {
      // ---- scores
      float sc[NT][4];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int e = 0; e < 4; ++e) sc[nt][e] = 0.f;
        if constexpr (BITS == 16) {
#pragma unroll
          for (int ks = 0; ks < D / 16; ++ks) mma<T>(sc[nt], qf[ks], kw[nt][2 * ks], kw[nt][2 * ks + 1]);
        } else if constexpr (BITS == 8) {
          const float zf = 8388608.f + static_cast<float>(kz[nt]);
#pragma unroll
          for (int ks = 0; ks < D / 16; ++ks) {
            const uint32_t w = kw[nt][ks];
            mma<T>(sc[nt], qf[ks], sub_pair8<T>(w, w, 0, 1, zf, zf), sub_pair8<T>(w, w, 2, 3, zf, zf));
          }
        } else {
          const uint32_t bias = bias4<T>(kz[nt], kz[nt]);
#pragma unroll
          for (int ks = 0; ks < D / 16; ++ks) {
            const uint32_t w = kw[nt][ks >> 1] >> ((ks & 1) * 8);
            mma<T>(sc[nt], qf[ks], sub_pair4<T>(w, bias), sub_pair4<T>(w >> 4, bias));
          }
        }
      }
      // ---- softmax: rows g and g + 8; a key that a row does not see weighs nothing, whatever it holds
      float mx[2] = {m[0], m[1]};
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float x = sc[nt][e] * a.scale_log2;
          if constexpr (BITS < 16) x *= (e & 1) ? ksc[nt].y : ksc[nt].x;
          x = k + nt * 8 + 2 * t + (e & 1) < see[e >> 1] ? x : -INFINITY;
          sc[nt][e] = x;
          mx[e >> 1] = fmaxf(mx[e >> 1], x);
        }
      if (k + STRIDE < k1) load_k(k + STRIDE, vecn);  // the keys' registers are free: next ones on their way
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        mx[r] = fmaxf(mx[r], __shfl_xor_sync(0xffffffffu, mx[r], 1));
        mx[r] = fmaxf(mx[r], __shfl_xor_sync(0xffffffffu, mx[r], 2));
      }
      if (__any_sync(0xffffffffu, mx[0] > m[0] || mx[1] > m[1])) {
        float corr[2];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          corr[r] = m[r] == -INFINITY ? 0.f : ex2(m[r] - mx[r]);
          l[r] *= corr[r];
          m[r] = mx[r];
        }
#pragma unroll
        for (int i = 0; i < NO; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[i][e] *= corr[e >> 1];
      }
      uint32_t pf[NT][2];  // [tile][row half]
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float p[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const bool sees = k + nt * 8 + 2 * t + (e & 1) < see[e >> 1];
          p[e] = sees ? ex2(sc[nt][e] - m[e >> 1]) : 0.f;
          l[e >> 1] += p[e];
          if constexpr (BITS < 16) p[e] = sees ? p[e] * ((e & 1) ? vsc[nt].y : vsc[nt].x) : 0.f;
        }
        pf[nt][0] = pack2<PT>(p[0], p[1]);
        pf[nt][1] = pack2<PT>(p[2], p[3]);
      }
      // a 16-bit value past the end of the keys must not meet its zero weight: it may be anything
      if constexpr (BITS == 16) {
        if (k + Y::KPW > k1) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int r = 0; r < 2; ++r)
              if (k + nt * 8 + 2 * t + r >= k1)
#pragma unroll
                for (int e = 0; e < Y::VW; ++e) vw[nt][r][e] = 0;
        }
      }
      // ---- weighted sum
#pragma unroll
      for (int kk = 0; kk < NT / 2; ++kk) {
        const uint32_t pa[4] = {pf[2 * kk][0], pf[2 * kk][1], pf[2 * kk + 1][0], pf[2 * kk + 1][1]};
        if constexpr (BITS == 16) {
#pragma unroll
          for (int w = 0; w < Y::VW; ++w)
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
              const uint32_t sel = hf ? 0x7632u : 0x5410u;
              mma<PT>(o[2 * w + hf], pa, __byte_perm(vw[2 * kk][0][w], vw[2 * kk][1][w], sel),
                      __byte_perm(vw[2 * kk + 1][0][w], vw[2 * kk + 1][1][w], sel));
            }
        } else if constexpr (BITS == 8) {
          float zf[2][2];
#pragma unroll
          for (int x = 0; x < 2; ++x)
#pragma unroll
            for (int r = 0; r < 2; ++r)
              zf[x][r] = 8388608.f + static_cast<float>((vz[2 * kk + x] >> (8 * r)) & 255);
#pragma unroll
          for (int w = 0; w < Y::VW; ++w)
#pragma unroll
            for (int b = 0; b < 4; ++b)
              mma<PT>(o[4 * w + b], pa, sub_pair8<PT>(vw[2 * kk][0][w], vw[2 * kk][1][w], b, b, zf[0][0], zf[0][1]),
                      sub_pair8<PT>(vw[2 * kk + 1][0][w], vw[2 * kk + 1][1][w], b, b, zf[1][0], zf[1][1]));
        } else {
          const uint32_t bz0 = bias4<PT>(vz[2 * kk] & 255, vz[2 * kk] >> 8);
          const uint32_t bz1 = bias4<PT>(vz[2 * kk + 1] & 255, vz[2 * kk + 1] >> 8);
#pragma unroll
          for (int w = 0; w < Y::VW; ++w)
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
              const uint32_t sel = hf ? 0x7632u : 0x5410u;
              const uint32_t x = __byte_perm(vw[2 * kk][0][w], vw[2 * kk][1][w], sel);
              const uint32_t y = __byte_perm(vw[2 * kk + 1][0][w], vw[2 * kk + 1][1][w], sel);
#pragma unroll
              for (int b = 0; b < 4; ++b)
                mma<PT>(o[8 * w + 4 * hf + b], pa, sub_pair4<PT>(x >> (4 * b), bz0), sub_pair4<PT>(y >> (4 * b), bz1));
            }
        }
      }
      if (k + STRIDE < k1) {
        load_v(k + STRIDE, vecn);
        find(k + 2 * STRIDE, vecn);
      }
    }
    // ---- the four warps' parts, then the piece
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
      l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
      if (t == 0) {
        red_m[warp * 16 + g + 8 * r] = m[r];
        red_l[warp * 16 + g + 8 * r] = l[r];
      }
#pragma unroll
      for (int c = 0; c < 2; ++c)
#pragma unroll
        for (int i = 0; i < NO; ++i)
          if (g + 8 * r < rows) red[(warp * 16 + g + 8 * r) * D + value_elem<D, BITS>(2 * t + c, i)] = o[i][2 * r + c];
    }
    __syncthreads();
    if constexpr (BITS == 16) {
      // Keys that some rows of the tile see and others do not: a value there that is not finite has met
      // the zero weight of a row that must not know it.  Such rows are done again, key by key.
      if (a.causal && k1 > q.len - q.n + 1) {
        for (int row = warp; row < rows; row += 4) {
          bool fine = true;
          for (int c = lane; c < 4 * D; c += 32) fine = fine && isfinite(red[((c / D) * 16 + row) * D + c % D]);
          if (__all_sync(0xffffffffu, fine)) continue;
          const int i = row / a.group;
          float rm, rl, acc[D / 32];
          row_attention<T, D, BITS>(a, s, h, qbase + (q.start + i) * a.q_ts + (h * a.group + row - i * a.group) * a.q_hs,
                                    k0, min(k1, seen(a, q, i)), rm, rl, acc);
          for (int w = 0; w < 4; ++w) {
            if (lane == 0) {
              red_m[w * 16 + row] = w ? -INFINITY : rm;
              red_l[w * 16 + row] = w ? 0.f : rl;
            }
#pragma unroll
            for (int c = 0; c < D / 32; ++c) red[(w * 16 + row) * D + lane + 32 * c] = w ? 0.f : acc[c];
          }
        }
        __syncthreads();
      }
    }
    const bool whole = cur.u0 == 0 && cur.u1 == cur.units;
    float* mine = whole ? nullptr : part + (static_cast<int64_t>(blockIdx.x) * 2 + (cur.at == first ? 0 : 1)) * step_part(D);
    for (int e = threadIdx.x; e < rows * (D / 4); e += ST_THREADS) {
      const int row = e / (D / 4), c = (e % (D / 4)) * 4;
      float mm = -INFINITY;
#pragma unroll
      for (int w = 0; w < 4; ++w) mm = fmaxf(mm, red_m[w * 16 + row]);
      const float ref = mm == -INFINITY ? 0.f : mm;
      float ll = 0.f;
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const float f = ex2(red_m[w * 16 + row] - ref);
        const float4 x = *reinterpret_cast<const float4*>(red + (w * 16 + row) * D + c);
        ll += f * red_l[w * 16 + row];
        v.x += f * x.x;
        v.y += f * x.y;
        v.z += f * x.z;
        v.w += f * x.w;
      }
      if (mine) {
        *reinterpret_cast<float4*>(mine + row * D + c) = v;
        if (c == 0) {
          mine[16 * D + row] = mm;
          mine[16 * D + 16 + row] = ll;
        }
      } else {
        const float inv = ll == 0.f ? 0.f : 1.f / ll;
        const int i = row / a.group;
        T* dst = static_cast<T*>(a.out) +
                 ((static_cast<int64_t>(q.start) + i) * a.heads + h * a.group + (row - i * a.group)) * D + c;
        uint2 w;
        w.x = pack2<T>(v.x * inv, v.y * inv);
        w.y = pack2<T>(v.z * inv, v.w * inv);
        *reinterpret_cast<uint2*>(dst) = w;
      }
    }
    __syncthreads();
  }
}

// Contexts of a few units are not cut: a piece per CTA, nothing to join.
constexpr int ST_WHOLE = 8;

template <typename T, int D, int BITS>
int run(const Args& a, int grid, bool cuts, float* part, Cut* cut, cudaStream_t s) {
  constexpr int smem = (4 * 16 * D + 2 * 4 * 16) * static_cast<int>(sizeof(float));
  GPTQ_TRY(ensure_smem_limit(reinterpret_cast<const void*>(step_kernel<T, D, BITS>), smem));
  Share sh;
  sh.whole = !cuts;
  sh.min_per = 4;
  sh.rows_lo = 1;
  sh.rows_hi = kStepRows;
  sh.grid = grid;
  step_kernel<T, D, BITS><<<grid, ST_THREADS, smem, s>>>(a, sh, part, cuts ? cut : nullptr);
  return after_launch();
}

}  // namespace

int step_grid(const Args& a, bool* cuts) {
  const int64_t units = ((a.table_width << a.page_shift) + ST_UNIT - 1) / ST_UNIT;
  const int64_t items = static_cast<int64_t>(a.seqs) * a.kv_heads;
  *cuts = units > ST_WHOLE;
  return static_cast<int>(*cuts ? std::min<int64_t>(items * units, 2 * num_sms()) : std::min<int64_t>(items, 1 << 20));
}

int run_step(const Args& a, int dtype, int head_dim, int bits, int grid, bool cuts, float* part, Cut* cut,
             cudaStream_t s) {
#define GPTQ_STEP(T, D)                                                                                        \
  return bits == 16  ? run<T, D, 16>(a, grid, cuts, part, cut, s)                                               \
         : bits == 8 ? run<T, D, 8>(a, grid, cuts, part, cut, s)                                                \
                     : run<T, D, 4>(a, grid, cuts, part, cut, s)
  if (dtype == GPTQ_BF16) {
    if (head_dim == 128) GPTQ_STEP(__nv_bfloat16, 128);
    GPTQ_STEP(__nv_bfloat16, 64);
  }
  if (head_dim == 128) GPTQ_STEP(__half, 128);
  GPTQ_STEP(__half, 64);
#undef GPTQ_STEP
}

}  // namespace paged
}  // namespace gptq
