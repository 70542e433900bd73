// Attention over a paged cache for sequences with few rows (at most 16 rows times heads of a kv
// head: single tokens, short guesses).
//
// Each key and value byte is used for at most 16 rows, so the cache's bytes bound the kernel and
// everything serves keeping loads in flight:
//  * The rows of all query heads that share a kv head are one 16-row tile (row i * group + g), so a
//    cache line is read once.  Scores and the weighted sum run on the 16x8x16 matrix instruction.
//  * Each warp has its own ring of steps in shared memory, filled by asynchronous copies two to seven steps
//    ahead (about 25 KB a warp, 200 KB an SM): the bytes in flight that the memory's latency asks for do not
//    fit in registers (prefetching there: 32 KB an SM, 8-bit cache at 3.4 TB/s).
//  * A lane's operands come from there without rearranging: the order of the contraction index is free as
//    long as both operands agree, so a lane takes contiguous 16-byte pieces of a key and the query is laid out
//    to match; for the values the column order is free, and a lane takes contiguous pieces of four keys.
//  * Codes enter the products as the float16 numbers 1024 + code (0x6400 | code: a byte permutation or one
//    logical operation per pair), and what that adds is taken off afterwards:
//      q . (c - z) = q . (1024 + c) - (1024 + z) sum(q),
//      sum_j w_j (c_j - z_j) = sum_j w_j (1024 + c_j) - sum_j w_j (1024 + z_j),
//    the last sum by one more column of the product.  (Both terms are exact products summed in fp32; their
//    difference keeps 2^-24 of 1280, against values of up to 255.)  A key's scale multiplies its scores, a
//    value's scale its probability: no value is rounded.  The query is brought into float16's range by a power
//    of two per row, and the weights w_j = p_j scale_j are held against their own running maximum, so that
//    float16 (2^-11) holds them whatever the scales are.  Subtracting zero points and rounding to 16 bits
//    pair by pair instead took 44 instructions per key and head of 128 and kept the cache's bytes waiting
//    (64 users, 8 bits: 196 us).
//  * The keys of all sequences are one line of 64-key units, cut into equal shares, one per resident
//    CTA: ragged lengths balance, and one long sequence fills the GPU.  A CTA's share has at most two
//    unfinished (sequence, head) pieces, its first and its last; those leave (maximum, sum, weighted
//    sum) behind and a second launch joins them in order, so results do not depend on timing.
// Each warp walks its own keys with its own running maximum and sum (fp32).
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
  static constexpr int CPR = ROW / 16;                     // 16-byte chunks of it
  static constexpr int KPW = BITS == 16 ? 16 : 32;         // keys of a warp's step
  static constexpr int NT = KPW / 8;                       // 8-key tiles of a step
  static constexpr int KP = KW >= 4 ? 4 : KW;              // words of a contiguous piece
  static constexpr int VP = VW >= 4 ? 4 : VW;
  // a warp's ring in shared memory: keys, values, and for codes their scales and zeros, of a step per stage
  static constexpr int SIDE = BITS == 16 ? 0 : KPW * 10;
  static constexpr int STAGE = 2 * KPW * ROW + SIDE;
  static constexpr int ROOM = 26624;                       // of a warp: 8 warps share an SM
  static constexpr int STAGES = ROOM / STAGE < 8 ? ROOM / STAGE : 8;
  static constexpr int PART = 16 * D * 4;                  // the warp's weighted sums afterwards
  static constexpr int RING = STAGES * STAGE > PART ? STAGES * STAGE : PART;
  // Chunk c of row r lies at chunk c ^ key_turn(r) (value_turn(r)) of its row, so that the 8 lanes that a 16-byte
  // read serves at once (two keys, four pieces; four values, two pieces) touch all banks.
  static __device__ __forceinline__ int key_turn(int r) { return CPR >= 8 ? (r & 1) << 2 : 0; }
  static __device__ __forceinline__ int value_turn(int r) { return CPR >= 8 ? r & 7 : (CPR == 4 ? (r >> 1) & 3 : 0); }
};

template <int N>
__device__ __forceinline__ void read_words(uint32_t at, uint32_t* w) {
  if constexpr (N == 4) {
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(at));
  } else if constexpr (N == 2) {
    asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(at));
  } else {
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(w[0]) : "r"(at));
  }
}

__device__ __forceinline__ uint32_t read_pair(uint32_t at) {  // two bytes
  uint16_t w;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(w) : "r"(at));
  return w;
}

__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
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

__device__ __forceinline__ float lg2(float x) {
  float y;
  asm("lg2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// 1024 + code of two codes as a pair of halves.
__device__ __forceinline__ uint32_t nibbles(uint32_t w) { return (w & 0x000f000fu) | 0x64006400u; }
__device__ __forceinline__ uint32_t low_bytes(uint32_t w) { return __byte_perm(w, 0x64646464u, 0x4140u); }
__device__ __forceinline__ uint32_t high_bytes(uint32_t w) { return __byte_perm(w, 0x64646464u, 0x4342u); }

template <typename T, int D, int BITS>
__global__ void __launch_bounds__(ST_THREADS, 2) step_kernel(const Args a, const Share sh, float* __restrict__ part, Cut* __restrict__ cut) {
  using Y = Lay<D, BITS>;
  using PT = typename std::conditional<BITS == 16, T, __half>::type;  // operands of the products
  constexpr int NT = Y::NT, NO = D / 8;
  extern __shared__ __align__(128) uint8_t smem[];  // a ring per warp, then maxima and sums
  float* red_m = reinterpret_cast<float*>(smem + 4 * Y::RING);
  float* red_l = red_m + 4 * 16;
  auto red = [&](int w, int row) { return reinterpret_cast<float*>(smem + w * Y::RING) + row * D; };
  __shared__ Cursor cur_s;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  next_may_start();

  Cursor cur;
  const bool any = first_piece<ST_THREADS>(a, sh, ST_UNIT, cur, &cur_s);
  if (cut && threadIdx.x == 0)
    cut[blockIdx.x] = any ? cut_at(cur.at, cur.per, cur.u0, cur.units, sequence(a, cur.s), cur.head, 0) : Cut{0, -1};
  if (!any) return;
  const int64_t first = cur.at;
  const uint32_t ring = static_cast<uint32_t>(__cvta_generic_to_shared(smem)) + warp * Y::RING;
  for (; cur.at < cur.end; next_piece(a, sh, ST_UNIT, cur)) {
    const Seq q = sequence(a, cur.s);
    const int rows = q.n * a.group;
    const int h = cur.head, s = cur.s;
    const int k0 = cur.u0 * ST_UNIT, k1 = min(cur.u1 * ST_UNIT, q.len);
    const T* qbase = static_cast<const T*>(a.q);
    const bool two = rows > 8;  // rows g + 8 are in use
    // keys seen by this lane's two rows; for codes: the row's power of two, and the sum of its query
    int see[2];
    float power[2] = {1.f, 1.f}, qsum[2] = {0.f, 0.f};
    uint32_t qf[D / 16][4];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int row = g + 8 * r;
      const bool in = row < rows;
      const int i = in ? row / a.group : 0;
      see[r] = in ? min(k1, seen(a, q, i)) : 0;
      const T* qr = qbase + (q.start + i) * a.q_ts + (h * a.group + (in ? row - i * a.group : 0)) * a.q_hs;
      uint4 raw[D / 32];  // 8 elements: two contraction steps
#pragma unroll
      for (int kk = 0; kk < D / 32; ++kk) {
        raw[kk] = make_uint4(0, 0, 0, 0);
        if (in) raw[kk] = __ldg(reinterpret_cast<const uint4*>(qr + key_elem<D, BITS>(t, kk)));
      }
      if constexpr (BITS < 16) {
        float top = 0.f;
#pragma unroll
        for (int kk = 0; kk < D / 32; ++kk)
#pragma unroll
          for (int e = 0; e < 8; ++e) top = fmaxf(top, fabsf(to_f32(reinterpret_cast<const T*>(&raw[kk])[e])));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const int ex = max(__float_as_int(top) >> 23, 1);  // biased exponent; infinity: NaN for the whole row
        const float down = ex < 255 ? __int_as_float((254 - ex) << 23) : __int_as_float(0x7fc00000);
        power[r] = __int_as_float(ex << 23);
        float sum = 0.f;
#pragma unroll
        for (int kk = 0; kk < D / 32; ++kk) {
          __half2 w[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const T* v = reinterpret_cast<const T*>(&raw[kk]) + 2 * e;
            w[e] = __floats2half2_rn(to_f32(v[0]) * down, to_f32(v[1]) * down);
            sum += __low2float(w[e]) + __high2float(w[e]);
          }
          raw[kk] = *reinterpret_cast<const uint4*>(w);
        }
        sum += __shfl_xor_sync(0xffffffffu, sum, 1);
        qsum[r] = sum + __shfl_xor_sync(0xffffffffu, sum, 2);
        power[r] *= a.scale_log2;
      }
#pragma unroll
      for (int kk = 0; kk < D / 32; ++kk) {
        const uint4 w = raw[kk];
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
    // for codes: running maximum of the weights (base 2), which the weighted sum is held against, and what the
    // codes' offsets add to it
    float mw[2] = {-INFINITY, -INFINITY}, off[4] = {0.f, 0.f, 0.f, 0.f};

    int64_t vecn[NT / 2];  // first vector of each 16 keys of the step to be loaded next
    auto find = [&](int k, int64_t (&v)[NT / 2]) {
#pragma unroll
      for (int j = 0; j < NT / 2; ++j) v[j] = k + 16 * j < k1 ? key_at(a, s, h, k + 16 * j) : 0;
    };
    // a step's copies: the 16 keys of a group are contiguous in their page, 16 bytes a lane; what lies past the
    // piece is not loaded
    auto load = [&](int k, int stage) {
      const uint32_t at = ring + stage * Y::STAGE;
#pragma unroll
      for (int j = 0; j < NT / 2; ++j) {
        if (k + 16 * j >= k1) continue;
        const uint8_t* ks = static_cast<const uint8_t*>(a.kc) + vecn[j] * Y::ROW + lane * 16;
        const uint8_t* vs = static_cast<const uint8_t*>(a.vc) + vecn[j] * Y::ROW + lane * 16;
#pragma unroll
        for (int x = 0; x < Y::CPR / 2; ++x) {
          const int r = x * (32 / Y::CPR) + lane / Y::CPR, c = lane % Y::CPR;
          const uint32_t row = at + (16 * j + r) * Y::ROW;
          copy16(row + ((c ^ Y::key_turn(r)) << 4), ks + x * 512);
          copy16(row + Y::KPW * Y::ROW + ((c ^ Y::value_turn(r)) << 4), vs + x * 512);
        }
        if constexpr (BITS < 16) {  // scales of keys and of values (64 bytes each), zeros (16 bytes each)
          const uint32_t side = at + 2 * Y::KPW * Y::ROW;
          if (lane < 8)
            copy16(side + ((lane >> 2) * Y::KPW + 16 * j) * 4 + (lane & 3) * 16,
                   ((lane & 4) ? a.vs : a.ks) + vecn[j] + (lane & 3) * 4);
          else if (lane < 10)
            copy16(side + 8 * Y::KPW + (lane - 8) * Y::KPW + 16 * j, ((lane & 1) ? a.vz : a.kz) + vecn[j]);
        }
      }
    };

    int k = k0 + warp * Y::KPW;
    constexpr int STRIDE = 4 * Y::KPW, AHEAD = Y::STAGES - 1;
    find(k, vecn);
#pragma unroll
    for (int x = 0; x < AHEAD; ++x) {
      if (k + x * STRIDE < k1) {
        load(k + x * STRIDE, x);
        find(k + (x + 1) * STRIDE, vecn);
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    }
    int stage = 0;
    for (; k < k1; k += STRIDE) {
      asm volatile("cp.async.wait_group %0;" ::"n"(AHEAD - 1) : "memory");
      __syncwarp();
      if (k + AHEAD * STRIDE < k1) {
        load(k + AHEAD * STRIDE, stage == 0 ? AHEAD : stage - 1);  // the stage that the last step has left
        find(k + (AHEAD + 1) * STRIDE, vecn);
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
      const uint32_t at = ring + stage * Y::STAGE, side = at + 2 * Y::KPW * Y::ROW;
      if (++stage == Y::STAGES) stage = 0;
      // ---- scores
      float sc[NT][4];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int e = 0; e < 4; ++e) sc[nt][e] = 0.f;
        uint32_t kw[Y::KW];
#pragma unroll
        for (int j = 0; j < Y::KW / Y::KP; ++j) {
          const int byte = (j * 4 + t) * Y::KP * 4;  // of the key's row
          read_words<Y::KP>(at + (nt * 8 + g) * Y::ROW + (((byte >> 4) ^ Y::key_turn(g)) << 4) + (byte & 15), kw + j * Y::KP);
        }
        if constexpr (BITS == 16) {
#pragma unroll
          for (int ks = 0; ks < D / 16; ++ks) mma<PT>(sc[nt], qf[ks], kw[2 * ks], kw[2 * ks + 1]);
        } else {
#pragma unroll
          for (int ks = 0; ks < D / 16; ++ks) {
            if constexpr (BITS == 8) {
              const uint32_t w = kw[ks];
              mma<PT>(sc[nt], qf[ks], low_bytes(w), high_bytes(w));
            } else {
              const uint32_t w = kw[ks >> 1] >> ((ks & 1) * 8);
              mma<PT>(sc[nt], qf[ks], nibbles(w), nibbles(w >> 4));
            }
          }
        }
      }
      // ---- softmax: rows g and g + 8; a key that a row does not see weighs nothing, whatever it holds
      float mx[2] = {m[0], m[1]}, mwx[2] = {mw[0], mw[1]};
      float lv[NT][2];   // log2 of the values' scales
      uint32_t vz[NT];  // their zeros, two bytes
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float zk[2], ks[2];
        if constexpr (BITS < 16) {  // of keys 2t, 2t + 1 of the tile
          uint32_t w[2];
          read_words<2>(side + 4 * (nt * 8 + 2 * t), w);
          ks[0] = __uint_as_float(w[0]);
          ks[1] = __uint_as_float(w[1]);
          read_words<2>(side + 4 * (Y::KPW + nt * 8 + 2 * t), w);
          lv[nt][0] = lg2(__uint_as_float(w[0]));
          lv[nt][1] = lg2(__uint_as_float(w[1]));
          const uint32_t z = read_pair(side + 8 * Y::KPW + nt * 8 + 2 * t);
          vz[nt] = read_pair(side + 9 * Y::KPW + nt * 8 + 2 * t);
          zk[0] = __uint_as_float(0x4B000000u | (z & 255u)) - 8387584.f;  // 2^23 - 1024: 1024 + zero
          zk[1] = __uint_as_float(0x4B000000u | (z >> 8)) - 8387584.f;
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if (e >= 2 && !two) continue;
          const int r = e >> 1, c = e & 1;
          float x;
          if constexpr (BITS < 16)
            x = fmaf(-zk[c], qsum[r], sc[nt][e]) * (ks[c] * power[r]);
          else
            x = sc[nt][e] * a.scale_log2;
          x = k + nt * 8 + 2 * t + c < see[r] ? x : -INFINITY;
          sc[nt][e] = x;
          mx[r] = fmaxf(mx[r], x);
          if constexpr (BITS < 16) mwx[r] = fmaxf(mwx[r], x + lv[nt][c]);
        }
      }
      bool grown = false;
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        if (r && !two) continue;
        mx[r] = fmaxf(mx[r], __shfl_xor_sync(0xffffffffu, mx[r], 1));
        mx[r] = fmaxf(mx[r], __shfl_xor_sync(0xffffffffu, mx[r], 2));
        grown = grown || mx[r] > m[r];
        if constexpr (BITS < 16) {
          mwx[r] = fmaxf(mwx[r], __shfl_xor_sync(0xffffffffu, mwx[r], 1));
          mwx[r] = fmaxf(mwx[r], __shfl_xor_sync(0xffffffffu, mwx[r], 2));
          grown = grown || mwx[r] > mw[r];
        }
      }
      if (__any_sync(0xffffffffu, grown)) {
        float corr[2];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          corr[r] = m[r] == -INFINITY ? 0.f : ex2(m[r] - mx[r]);
          l[r] *= corr[r];
          m[r] = mx[r];
          if constexpr (BITS < 16) {
            corr[r] = mw[r] == -INFINITY ? 0.f : ex2(mw[r] - mwx[r]);
            mw[r] = mwx[r];
            off[2 * r] *= corr[r];
          }
        }
#pragma unroll
        for (int i = 0; i < NO; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[i][e] *= corr[e >> 1];
      }
      uint32_t pf[NT][2];  // [tile][row half]
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float p[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if (e >= 2 && !two) continue;
          const int r = e >> 1;
          const bool sees = k + nt * 8 + 2 * t + (e & 1) < see[r];
          p[e] = sees ? ex2(sc[nt][e] - m[r]) : 0.f;
          l[r] += p[e];
          if constexpr (BITS < 16) {
            const float ref = mw[r] == -INFINITY ? 0.f : mw[r];  // scales of zero alone so far
            p[e] = sees ? ex2(sc[nt][e] + lv[nt][e & 1] - ref) : 0.f;
          }
        }
        pf[nt][0] = pack2<PT>(p[0], p[1]);
        pf[nt][1] = pack2<PT>(p[2], p[3]);
      }
      // ---- weighted sum
#pragma unroll
      for (int kk = 0; kk < NT / 2; ++kk) {
        const uint32_t pa[4] = {pf[2 * kk][0], pf[2 * kk][1], pf[2 * kk + 1][0], pf[2 * kk + 1][1]};
        uint32_t vw[2][2][Y::VW];  // [8-key tile][key 2t, 2t + 1]
#pragma unroll
        for (int x = 0; x < 2; ++x)
#pragma unroll
          for (int r = 0; r < 2; ++r) {
#pragma unroll
            for (int j = 0; j < Y::VW / Y::VP; ++j) {
              const int byte = (j * 8 + g) * Y::VP * 4;
              read_words<Y::VP>(at + (Y::KPW + (2 * kk + x) * 8 + 2 * t + r) * Y::ROW +
                                    (((byte >> 4) ^ Y::value_turn(2 * t + r)) << 4) + (byte & 15),
                                vw[x][r] + j * Y::VP);
            }
            // a 16-bit value past the end of the keys must not meet its zero weight: it may be anything
            if (BITS == 16 && k + Y::KPW > k1 && k + (2 * kk + x) * 8 + 2 * t + r >= k1) {
#pragma unroll
              for (int e = 0; e < Y::VW; ++e) vw[x][r][e] = 0;
            }
          }
        if constexpr (BITS == 16) {
#pragma unroll
          for (int w = 0; w < Y::VW; ++w)
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
              const uint32_t sel = hf ? 0x7632u : 0x5410u;
              mma<PT>(o[2 * w + hf], pa, __byte_perm(vw[0][0][w], vw[0][1][w], sel),
                      __byte_perm(vw[1][0][w], vw[1][1][w], sel));
            }
        } else {
          // the offsets' column: 1024 + zero of the four keys
          mma<PT>(off, pa, low_bytes(vz[2 * kk]), low_bytes(vz[2 * kk + 1]));
#pragma unroll
          for (int w = 0; w < Y::VW; ++w) {
            const uint32_t a0 = vw[0][0][w], a1 = vw[0][1][w];
            const uint32_t b0 = vw[1][0][w], b1 = vw[1][1][w];
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
              if constexpr (BITS == 8) {
                const uint32_t sel = hf ? 0x7362u : 0x5140u;  // bytes 2 hf, 2 hf + 1 of both keys
                const uint32_t x = __byte_perm(a0, a1, sel), y = __byte_perm(b0, b1, sel);
                mma<PT>(o[4 * w + 2 * hf], pa, low_bytes(x), low_bytes(y));
                mma<PT>(o[4 * w + 2 * hf + 1], pa, high_bytes(x), high_bytes(y));
              } else {
                const uint32_t sel = hf ? 0x7632u : 0x5410u;
                const uint32_t x = __byte_perm(a0, a1, sel), y = __byte_perm(b0, b1, sel);
#pragma unroll
                for (int b = 0; b < 4; ++b) mma<PT>(o[8 * w + 4 * hf + b], pa, nibbles(x >> (4 * b)), nibbles(y >> (4 * b)));
              }
            }
          }
        }
      }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncwarp();
    // ---- the four warps' parts, then the piece
    if constexpr (BITS < 16) {
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const float f = mw[r] == -INFINITY ? 0.f : ex2(mw[r] - m[r]);
#pragma unroll
        for (int i = 0; i < NO; ++i)
#pragma unroll
          for (int c = 0; c < 2; ++c) o[i][2 * r + c] = (o[i][2 * r + c] - off[2 * r]) * f;
      }
    }
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
          if (g + 8 * r < rows) red(warp, g + 8 * r)[value_elem<D, BITS>(2 * t + c, i)] = o[i][2 * r + c];
    }
    __syncthreads();
    if constexpr (BITS == 16) {
      // Keys that some rows of the tile see and others do not: a value there that is not finite has met
      // the zero weight of a row that must not know it.  Such rows are done again, key by key.
      if (a.causal && k1 > q.len - q.n + 1) {
        for (int row = warp; row < rows; row += 4) {
          bool fine = true;
          for (int c = lane; c < 4 * D; c += 32) fine = fine && isfinite(red(c / D, row)[c % D]);
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
            for (int c = 0; c < D / 32; ++c) red(w, row)[lane + 32 * c] = w ? 0.f : acc[c];
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
        const float4 x = *reinterpret_cast<const float4*>(red(w, row) + c);
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
  constexpr int smem = 4 * Lay<D, BITS>::RING + 2 * 4 * 16 * static_cast<int>(sizeof(float));
  static_assert(2 * (smem + 1024 + 512) <= 233472, "two CTAs share an SM");
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
