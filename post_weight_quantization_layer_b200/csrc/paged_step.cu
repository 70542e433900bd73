// Attention over a paged cache for sequences with few rows (at most 16 rows times heads of a kv
// head: single tokens, short guesses).
//
// Each key and value byte is used for at most 16 rows, so the cache's bytes bound the kernel, and after
// them the instructions that codes take (4 bits: half the bytes, the same instructions):
//  * The rows of all query heads that share a kv head (row i * group + g) are the 8 (or 2 x 8) columns of the
//    16x8x16 matrix instruction, keys, and then the columns of the values, its 16 rows: a cache line is read
//    once, and up to 8 rows cost half the products and accumulators of a 16-row tile (64 users of 70B-shaped
//    heads, 8 bits: 148 -> 118 us; four users, 131072 keys, 4 bits: 249 -> 183 us; as it stands 115 and 186 from a
//    graph that replays one input, 132 and 190 among calls with others).
//  * Each warp has its own ring of steps in shared memory, filled by asynchronous copies one to seven steps
//    ahead (17 KB a warp, 200 KB an SM): the bytes in flight that the memory's latency asks for do not fit in
//    registers (prefetching there: 32 KB an SM, 8-bit cache at 3.4 TB/s; now 5.4).
//  * A lane's operands come from there without rearranging: the order of the contraction index is free as
//    long as both operands agree, so a lane takes contiguous 16-byte pieces of a key and the query is laid out
//    to match; for the values the column order is free, and a lane takes contiguous pieces of four keys.  The
//    probabilities are turned into an operand by a transposition across the warp.
//  * Codes enter the products as float16 numbers: exact, and without a conversion of their own (1024 + code
//    is 0x6400 | code, 64 + code of a nibble in bits 4-7 is 0x5400 | bits: a byte permutation or one logical
//    operation per pair).  Values have 1024 + zero subtracted (exactly) before they are multiplied: their sum over
//    a long context is small, and an offset taken off after it left 0.39 of it wrong at 131072 keys of 4 bits.
//    Keys keep their offset, which a contraction over one head affords: q . (c - z) = q . (o + c) - (o + z) sum(q).
//    A key's scale multiplies its scores, a value's scale its probability: no value is rounded.  The query is
//    brought to the upper end of float16's range by a power of two per row, and the weights w_j = p_j scale_j are
//    held against their own running maximum, so that float16 (2^-11) holds them whatever the scales are.
//    (Converting pair by pair to 16 bits through fp32: 44 instructions per key and head of 128.)
//  * The keys of all sequences are one line of 64-key units, cut into equal shares, one per resident
//    CTA: ragged lengths balance, and one long sequence fills the GPU.  A CTA's share has at most two
//    unfinished (sequence, head) pieces, its first and its last; those leave (maximum, sum, weighted
//    sum) behind and a second launch joins them in order, so results do not depend on timing.
//  * Few items of short contexts go to clusters of CTAs instead, an item each, which join through shared
//    memory in the same launch (one user, 32 heads, 2500 keys: 16.2 -> 11.7 us, 12.7 among calls with other inputs; its
//    bytes take 6.4).
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
template <int D, int BITS, int NR>
struct Lay {
  static constexpr int KW = D / 4 * BITS / 32;
  static constexpr int VW = D / 8 * BITS / 32;
  static constexpr int ROW = D * BITS / 8;                 // bytes of a vector
  static constexpr int CPR = ROW / 16;                     // 16-byte chunks of it
  static constexpr int KPW = BITS == 4 ? 32 : 16;          // keys of a warp's step
  static constexpr int NK = KPW / 16;                      // 16-key groups of it
  static constexpr int KP = KW >= 4 ? 4 : KW;              // words of a contiguous piece
  static constexpr int VP = VW >= 4 ? 4 : VW;
  // a warp's ring in shared memory: keys, values, and for codes their scales and zeros, of a step per stage
  static constexpr int SIDE = BITS == 16 ? 0 : KPW * 10;
  static constexpr int STAGE = 2 * KPW * ROW + SIDE;
  static constexpr int CTAS = NR == 2 ? 2 : 3;            // of an SM
  static constexpr int ROOM = CTAS == 2 ? 26624 : 17920;   // of a warp
  static constexpr int STAGES = ROOM / STAGE < 8 ? ROOM / STAGE : 8;
  static constexpr int PART = 8 * NR * D * 4;              // the warp's weighted sums afterwards
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

__device__ __forceinline__ uint32_t read_byte(uint32_t at) {
  uint16_t w;
  asm volatile("ld.shared.u8 %0, [%1];" : "=h"(w) : "r"(at));
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

// Codes as pairs of halves: 1024 + code of bytes, 64 + code of nibbles in bits 4-7 of each half (keys); of
// values 1024 + code, or 1024 + 16 code for the upper nibbles of a byte, which come without a shift.
__device__ __forceinline__ uint32_t low_bytes(uint32_t w) { return __byte_perm(w, 0x64646464u, 0x4140u); }
__device__ __forceinline__ uint32_t high_bytes(uint32_t w) { return __byte_perm(w, 0x64646464u, 0x4342u); }
__device__ __forceinline__ uint32_t key_nibbles(uint32_t w) { return (w & 0x00f000f0u) | 0x54005400u; }
__device__ __forceinline__ uint32_t low_nibbles(uint32_t w) { return (w & 0x000f000fu) | 0x64006400u; }
__device__ __forceinline__ uint32_t high_nibbles(uint32_t w) { return (w & 0x00f000f0u) | 0x64006400u; }
__device__ __forceinline__ uint32_t less(uint32_t a, uint32_t b) {
  const __half2 d = __hsub2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
  return *reinterpret_cast<const uint32_t*>(&d);
}

// The shared memory of the CTAs of a cluster.  Threads of a warp come here from loops that some of them leave
// earlier (heads of 64 and an odd number of rows), so the barrier is the form that asks no convergence of them.
__device__ __forceinline__ void team_barrier() {
  asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}
__device__ __forceinline__ uint32_t peer(uint32_t at, int rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(at), "r"(rank));
  return r;
}
__device__ __forceinline__ float peer_float(uint32_t at) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(at) : "memory");
  return v;
}
__device__ __forceinline__ float4 peer_float4(uint32_t at) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(at) : "memory");
  return v;
}

// An 8 x 8 matrix of 16-bit values, a row of pairs per four lanes, turned round.
__device__ __forceinline__ uint32_t turned(uint32_t w) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(w));
  return r;
}

template <typename T, int D, int BITS, int NR>
__global__ void __launch_bounds__(ST_THREADS, (Lay<D, BITS, NR>::CTAS))
    step_kernel(const Args a, const Share sh, float* __restrict__ part, Cut* __restrict__ cut) {
  using Y = Lay<D, BITS, NR>;
  using PT = typename std::conditional<BITS == 16, T, __half>::type;  // operands of the products
  constexpr int NK = Y::NK, NO = D / 16;
  // Weights in float16 are held against 2^15, not 1: many keys that weigh under 2^-25 of the largest, float16's last
  // step, may count for something together.
  constexpr float UP = std::is_same<PT, __half>::value ? 15.f : 0.f;
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
    // The products have keys (or values' columns) as their 16 rows and 8 rows of the sequence as their columns:
    // a lane holds the query of row g (of each 8) as an operand and the scores of rows 2t, 2t + 1.
    uint32_t qf[NR][D / 16][2];
    int see[NR][2], least = k1;
    float power[NR][2], qsum[NR][2];  // for codes: see below
#pragma unroll
    for (int r = 0; r < NR; ++r) {
      const int row = 8 * r + g;
      const bool in = row < rows;
      const int i = in ? row / a.group : 0;
      const int mine = in ? min(k1, seen(a, q, i)) : 0;
      least = min(least, in ? mine : k1);
      const T* qr = qbase + (q.start + i) * a.q_ts + (h * a.group + (in ? row - i * a.group : 0)) * a.q_hs;
      uint4 raw[D / 32];  // 8 elements: two contraction steps
#pragma unroll
      for (int kk = 0; kk < D / 32; ++kk) {
        raw[kk] = make_uint4(0, 0, 0, 0);
        if (in) raw[kk] = __ldg(reinterpret_cast<const uint4*>(qr + key_elem<D, BITS>(t, kk)));
      }
      float up = 1.f, sum = 0.f;
      if constexpr (BITS < 16) {
        // the row over a power of two, its largest in 2^14 .. 2^15 of float16 (elements down to 2^-28 of it keep all
        // their bits; the sums of 128 products with codes stay below 2^33), and its sum
        float top = 0.f;
#pragma unroll
        for (int kk = 0; kk < D / 32; ++kk)
#pragma unroll
          for (int e = 0; e < 8; ++e) top = fmaxf(top, fabsf(to_f32(reinterpret_cast<const T*>(&raw[kk])[e])));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const int ex = max(__float_as_int(top) >> 23, 15);  // biased exponent; infinity: NaN for the whole row
        const float down = ex < 255 ? __int_as_float((254 + 14 - ex) << 23) : __int_as_float(0x7fc00000);
        up = __int_as_float((ex - 14) << 23) * a.scale_log2;
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
        sum += __shfl_xor_sync(0xffffffffu, sum, 2);
      }
#pragma unroll
      for (int kk = 0; kk < D / 32; ++kk) {
        const uint4 w = raw[kk];
        if constexpr (BITS == 4) {  // pairs (e, e + 4), as the codes' nibbles come out
          qf[r][2 * kk][0] = __byte_perm(w.x, w.z, 0x5410);
          qf[r][2 * kk][1] = __byte_perm(w.x, w.z, 0x7632);
          qf[r][2 * kk + 1][0] = __byte_perm(w.y, w.w, 0x5410);
          qf[r][2 * kk + 1][1] = __byte_perm(w.y, w.w, 0x7632);
        } else {
          qf[r][2 * kk][0] = w.x;
          qf[r][2 * kk][1] = w.y;
          qf[r][2 * kk + 1][0] = w.z;
          qf[r][2 * kk + 1][1] = w.w;
        }
      }
#pragma unroll
      for (int c = 0; c < 2; ++c) {  // from the lanes that hold rows 2t, 2t + 1
        const int from = (2 * t + c) * 4;
        see[r][c] = __shfl_sync(0xffffffffu, mine, from);
        if constexpr (BITS < 16) {
          power[r][c] = __shfl_sync(0xffffffffu, up, from);
          qsum[r][c] = __shfl_sync(0xffffffffu, sum, from);
        }
      }
    }
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) least = min(least, __shfl_xor_sync(0xffffffffu, least, o));
    float o[NR][NO][4];
#pragma unroll
    for (int r = 0; r < NR; ++r)
#pragma unroll
      for (int i = 0; i < NO; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[r][i][e] = 0.f;
    // Running maximum and sum.  For codes also the running maximum of the weights (base 2), which the weighted
    // sum is held against.
    float m[NR][2], l[NR][2], mw[NR][2];
#pragma unroll
    for (int r = 0; r < NR; ++r) {
      m[r][0] = m[r][1] = mw[r][0] = mw[r][1] = -INFINITY;
      l[r][0] = l[r][1] = 0.f;
    }

    int64_t vecn[NK];  // first vector of each 16 keys of the step to be loaded next
    auto find = [&](int k, int64_t (&v)[NK]) {
#pragma unroll
      for (int j = 0; j < NK; ++j) v[j] = k + 16 * j < k1 ? key_at(a, s, h, k + 16 * j) : 0;
    };
    // a step's copies: the 16 keys of a group are contiguous in their page, 16 bytes a lane; what lies past the
    // piece is not loaded
    auto load = [&](int k, int stage) {
      const uint32_t at = ring + stage * Y::STAGE;
#pragma unroll
      for (int j = 0; j < NK; ++j) {
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
      // ---- scores, 16 keys at a time: a lane gets those of keys g, g + 8 and rows 2t, 2t + 1
      float sc[NK][NR][4], lv[NK][2];  // scores (base 2), log2 of the values' scales
      uint32_t vz[NK][2];              // values' zeros of keys 2t, 2t + 1 and 2t + 8, 2t + 9
      float mx[NR][2], mwx[NR][2];
#pragma unroll
      for (int r = 0; r < NR; ++r)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          mx[r][c] = m[r][c];
          mwx[r][c] = mw[r][c];
        }
      const bool all = k + Y::KPW <= least;  // every row sees every key of the step
#pragma unroll
      for (int kk = 0; kk < NK; ++kk) {
        uint32_t ka[Y::KW], kb[Y::KW];
#pragma unroll
        for (int j = 0; j < Y::KW / Y::KP; ++j) {
          const int byte = (j * 4 + t) * Y::KP * 4;  // of the key's row
          const uint32_t from = at + (kk * 16 + g) * Y::ROW + (((byte >> 4) ^ Y::key_turn(g)) << 4) + (byte & 15);
          read_words<Y::KP>(from, ka + j * Y::KP);
          read_words<Y::KP>(from + 8 * Y::ROW, kb + j * Y::KP);
        }
#pragma unroll
        for (int r = 0; r < NR; ++r)
#pragma unroll
          for (int e = 0; e < 4; ++e) sc[kk][r][e] = BITS < 16 ? (BITS == 8 ? -1024.f : -64.f) * qsum[r][e & 1] : 0.f;
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
          uint32_t f[4];
          if constexpr (BITS == 16) {
            f[0] = ka[2 * ks];
            f[1] = kb[2 * ks];
            f[2] = ka[2 * ks + 1];
            f[3] = kb[2 * ks + 1];
          } else if constexpr (BITS == 8) {
            f[0] = low_bytes(ka[ks]);
            f[1] = low_bytes(kb[ks]);
            f[2] = high_bytes(ka[ks]);
            f[3] = high_bytes(kb[ks]);
          } else {
            const uint32_t x = ka[ks >> 1], y = kb[ks >> 1];
            f[0] = key_nibbles((ks & 1) ? x >> 4 : x << 4);
            f[1] = key_nibbles((ks & 1) ? y >> 4 : y << 4);
            f[2] = key_nibbles((ks & 1) ? x >> 8 : x);
            f[3] = key_nibbles((ks & 1) ? y >> 8 : y);
          }
#pragma unroll
          for (int r = 0; r < NR; ++r) mma<PT>(sc[kk][r], f, qf[r][ks][0], qf[r][ks][1]);
        }
        float scale[2], zero[2];
        if constexpr (BITS < 16) {
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const int key = kk * 16 + 8 * x + g;
            uint32_t w;
            read_words<1>(side + 4 * key, &w);
            scale[x] = __uint_as_float(w);
            read_words<1>(side + 4 * (Y::KPW + key), &w);
            lv[kk][x] = lg2(__uint_as_float(w));
            zero[x] = __uint_as_float(0x4B000000u | read_byte(side + 8 * Y::KPW + key)) - 8388608.f;
            vz[kk][x] = read_pair(side + 9 * Y::KPW + kk * 16 + 8 * x + 2 * t);
          }
        }
#pragma unroll
        for (int r = 0; r < NR; ++r)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float x = sc[kk][r][e];
            if constexpr (BITS < 16)
              x = fmaf(-zero[e >> 1], qsum[r][e & 1], x) * (scale[e >> 1] * power[r][e & 1]);
            else
              x *= a.scale_log2;
            // a key that a row does not see weighs nothing, whatever it holds
            if (!all && k + kk * 16 + 8 * (e >> 1) + g >= see[r][e & 1]) x = -INFINITY;
            sc[kk][r][e] = x;
            mx[r][e & 1] = fmaxf(mx[r][e & 1], x);
            if constexpr (BITS < 16) mwx[r][e & 1] = fmaxf(mwx[r][e & 1], x + lv[kk][e >> 1]);
          }
      }
      // ---- softmax
      bool grown = false;
#pragma unroll
      for (int r = 0; r < NR; ++r)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
#pragma unroll
          for (int x = 4; x < 32; x <<= 1) mx[r][c] = fmaxf(mx[r][c], __shfl_xor_sync(0xffffffffu, mx[r][c], x));
          grown = grown || mx[r][c] > m[r][c];
          if constexpr (BITS < 16) {
#pragma unroll
            for (int x = 4; x < 32; x <<= 1) mwx[r][c] = fmaxf(mwx[r][c], __shfl_xor_sync(0xffffffffu, mwx[r][c], x));
            grown = grown || mwx[r][c] > mw[r][c];
          }
        }
      if (__any_sync(0xffffffffu, grown)) {
#pragma unroll
        for (int r = 0; r < NR; ++r)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            float f = m[r][c] == -INFINITY ? 0.f : ex2(m[r][c] - mx[r][c]);
            l[r][c] *= f;
            m[r][c] = mx[r][c];
            if constexpr (BITS < 16) {
              f = mw[r][c] == -INFINITY ? 0.f : ex2(mw[r][c] - mwx[r][c]);
              mw[r][c] = mwx[r][c];
            }
#pragma unroll
            for (int i = 0; i < NO; ++i) {
              o[r][i][c] *= f;
              o[r][i][2 + c] *= f;
            }
          }
      }
      uint32_t pf[NK][NR][2];
#pragma unroll
      for (int kk = 0; kk < NK; ++kk)
#pragma unroll
        for (int r = 0; r < NR; ++r) {
          float p[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int c = e & 1;
            const bool sees = all || k + kk * 16 + 8 * (e >> 1) + g < see[r][c];
            const float top = m[r][c] == -INFINITY ? 0.f : m[r][c];  // scores of -infinity alone so far: weights of 0
            p[e] = sees ? ex2(sc[kk][r][e] - (BITS == 16 ? top - UP : top)) : 0.f;
            l[r][c] += p[e];
            if constexpr (BITS < 16) {
              const float ref = mw[r][c] == -INFINITY ? 0.f : mw[r][c];  // scales of zero alone so far
              p[e] = sees ? ex2(sc[kk][r][e] + lv[kk][e >> 1] - (ref - UP)) : 0.f;
            }
          }
          pf[kk][r][0] = turned(pack2<PT>(p[0], p[1]));
          pf[kk][r][1] = turned(pack2<PT>(p[2], p[3]));
        }
      // ---- weighted sum: columns of the values (two of a lane's) by 16 keys
#pragma unroll
      for (int kk = 0; kk < NK; ++kk) {
        uint32_t vw[2][2][Y::VW];  // [8-key tile][key 2t, 2t + 1]
#pragma unroll
        for (int x = 0; x < 2; ++x)
#pragma unroll
          for (int r = 0; r < 2; ++r) {
#pragma unroll
            for (int j = 0; j < Y::VW / Y::VP; ++j) {
              const int byte = (j * 8 + g) * Y::VP * 4;
              read_words<Y::VP>(at + (Y::KPW + kk * 16 + x * 8 + 2 * t + r) * Y::ROW +
                                    (((byte >> 4) ^ Y::value_turn(2 * t + r)) << 4) + (byte & 15),
                                vw[x][r] + j * Y::VP);
            }
            // a 16-bit value past the end of the keys must not meet its zero weight: it may be anything
            if (BITS == 16 && k + Y::KPW > k1 && k + kk * 16 + x * 8 + 2 * t + r >= k1) {
#pragma unroll
              for (int e = 0; e < Y::VW; ++e) vw[x][r][e] = 0;
            }
          }
        // 1024 + zero of the four keys, and 1024 + 16 zero
        uint32_t z0 = 0, z1 = 0, y0 = 0, y1 = 0;
        if constexpr (BITS < 16) {
          z0 = low_bytes(vz[kk][0]);
          z1 = low_bytes(vz[kk][1]);
          y0 = ((z0 & 0x000f000fu) << 4) | 0x64006400u;
          y1 = ((z1 & 0x000f000fu) << 4) | 0x64006400u;
        }
        auto add = [&](int i, uint32_t f0, uint32_t f1, uint32_t f2, uint32_t f3) {
          const uint32_t f[4] = {f0, f1, f2, f3};
#pragma unroll
          for (int r = 0; r < NR; ++r) mma<PT>(o[r][i], f, pf[kk][r][0], pf[kk][r][1]);
        };
#pragma unroll
        for (int w = 0; w < Y::VW; ++w) {
          const uint32_t a0 = vw[0][0][w], a1 = vw[0][1][w], b0 = vw[1][0][w], b1 = vw[1][1][w];
          if constexpr (BITS == 16) {
            add(w, __byte_perm(a0, a1, 0x5410u), __byte_perm(a0, a1, 0x7632u), __byte_perm(b0, b1, 0x5410u),
                __byte_perm(b0, b1, 0x7632u));
          } else {
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
              if constexpr (BITS == 8) {
                const uint32_t sel = hf ? 0x7362u : 0x5140u;  // bytes 2 hf, 2 hf + 1 of both keys
                const uint32_t x = __byte_perm(a0, a1, sel), y = __byte_perm(b0, b1, sel);
                add(2 * w + hf, less(low_bytes(x), z0), less(high_bytes(x), z0), less(low_bytes(y), z1), less(high_bytes(y), z1));
              } else {
                const uint32_t sel = hf ? 0x7632u : 0x5410u;
                const uint32_t x = __byte_perm(a0, a1, sel), y = __byte_perm(b0, b1, sel);
#pragma unroll
                for (int b = 0; b < 2; ++b)
                  add(4 * w + 2 * hf + b, less(low_nibbles(x >> (8 * b)), z0), less(high_nibbles(x >> (8 * b)), y0),
                      less(low_nibbles(y >> (8 * b)), z1), less(high_nibbles(y >> (8 * b)), y1));
              }
            }
          }
        }
      }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncwarp();
    // ---- the four warps' parts, then the piece
#pragma unroll
    for (int r = 0; r < NR; ++r)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int row = 8 * r + 2 * t + c;
        if constexpr (BITS < 16) {  // back to the row's own maximum; upper nibbles came 16 times as large
          // the factor by its root: of small values it may be below float32's range when the product is not
          const float f = mw[r][c] == -INFINITY ? 0.f : ex2(0.5f * (mw[r][c] - UP - m[r][c]));
#pragma unroll
          for (int i = 0; i < NO; ++i) {
            o[r][i][c] = o[r][i][c] * f * f;
            o[r][i][2 + c] = o[r][i][2 + c] * (BITS == 4 ? f * 0.0625f : f) * f;
          }
        }
#pragma unroll
        for (int x = 4; x < 32; x <<= 1) l[r][c] += __shfl_xor_sync(0xffffffffu, l[r][c], x);
        if (g == 0) {
          red_m[warp * 16 + row] = BITS == 16 ? m[r][c] - UP : m[r][c];  // what sums and results are held against
          red_l[warp * 16 + row] = l[r][c];
        }
        if (row < rows) {
#pragma unroll
          for (int i = 0; i < NO; ++i)
#pragma unroll
            for (int x = 0; x < 2; ++x) red(warp, row)[value_elem<D, BITS>(g, 2 * i + x)] = o[r][i][2 * x + c];
        }
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
    const bool whole = sh.whole || (cur.u0 == 0 && cur.u1 == cur.units);
    const int team = sh.whole ? sh.whole : 1;
    float* both = reinterpret_cast<float*>(smem + Y::PART);  // this CTA's part, for its team
    float* mine = team > 1 ? both : whole ? nullptr : part + (static_cast<int64_t>(blockIdx.x) * 2 + (cur.at == first ? 0 : 1)) * step_part(D);
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
          mine[kStepRows * D + row] = mm;
          mine[kStepRows * (D + 1) + row] = ll;
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
    if (team > 1) {
      // The team's parts, read from the shared memory of its CTAs, each of which joins its share of the columns, in
      // the order of the keys.
      team_barrier();
      const int rank = blockIdx.x % team;
      const uint32_t from = static_cast<uint32_t>(__cvta_generic_to_shared(both));
      for (int e = rank * ST_THREADS + threadIdx.x; e < rows * (D / 4); e += team * ST_THREADS) {
        const int row = e / (D / 4), c = (e % (D / 4)) * 4;
        float pm[8], pl[8];
        float4 y[8];
#pragma unroll
        for (int x = 0; x < 8; ++x) {
          pm[x] = -INFINITY;
          pl[x] = 0.f;
          y[x] = make_float4(0.f, 0.f, 0.f, 0.f);
          if (x >= team) continue;
          const uint32_t there = peer(from, x);
          pm[x] = peer_float(there + (kStepRows * D + row) * 4);
          pl[x] = peer_float(there + (kStepRows * (D + 1) + row) * 4);
          y[x] = peer_float4(there + (row * D + c) * 4);
        }
        float mm = -INFINITY, ll = 0.f;
#pragma unroll
        for (int x = 0; x < 8; ++x) mm = fmaxf(mm, pm[x]);
        const float ref = mm == -INFINITY ? 0.f : mm;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int x = 0; x < 8; ++x) {
          if (x >= team) continue;
          const float f = ex2(pm[x] - ref);
          ll += f * pl[x];
          v.x += f * y[x].x;
          v.y += f * y[x].y;
          v.z += f * y[x].z;
          v.w += f * y[x].w;
        }
        const float inv = ll == 0.f ? 0.f : 1.f / ll;
        const int i = row / a.group;
        T* dst = static_cast<T*>(a.out) +
                 ((static_cast<int64_t>(q.start) + i) * a.heads + h * a.group + (row - i * a.group)) * D + c;
        uint2 w;
        w.x = pack2<T>(v.x * inv, v.y * inv);
        w.y = pack2<T>(v.z * inv, v.w * inv);
        *reinterpret_cast<uint2*>(dst) = w;
      }
      team_barrier();  // nobody leaves, or goes on, while its part is read
    }
    __syncthreads();
  }
}

// No sequence of the call has more than 8 rows here: half the products and registers.
bool eight(const Args& a) { return static_cast<int64_t>(a.max_q) * a.group <= 8; }

template <typename T, int D, int BITS, int NR>
int run(const Args& a, int grid, int team, float* part, Cut* cut, cudaStream_t s) {
  using Y = Lay<D, BITS, NR>;
  constexpr int smem = 4 * Y::RING + 2 * 4 * 16 * static_cast<int>(sizeof(float));
  static_assert(Y::STAGES >= 2 && Y::CTAS * (smem + 1024 + 256) <= 233472, "the CTAs of an SM share its memory");
  GPTQ_TRY(ensure_smem_limit(reinterpret_cast<const void*>(step_kernel<T, D, BITS, NR>), smem));
  Share sh;
  sh.whole = team;
  sh.min_per = 4;
  sh.rows_lo = 1;
  sh.rows_hi = kStepRows;
  sh.grid = grid;
  static_assert(Y::PART + step_part(D) * 4 <= Y::RING, "a team's parts lie behind the first warp's");
  if (team > 1) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(ST_THREADS);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = team;
    at[0].val.clusterDim.y = 1;
    at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, step_kernel<T, D, BITS, NR>, a, sh, part, static_cast<Cut*>(nullptr)) != cudaSuccess) {
      cudaGetLastError();
      return GPTQ_ERR_CUDA;
    }
    return after_launch();
  }
  step_kernel<T, D, BITS, NR><<<grid, ST_THREADS, smem, s>>>(a, sh, part, team == 0 ? cut : nullptr);
  return after_launch();
}

template <typename T, int D, int BITS>
int run(const Args& a, int grid, int team, float* part, Cut* cut, cudaStream_t s) {
  return eight(a) ? run<T, D, BITS, 1>(a, grid, team, part, cut, s) : run<T, D, BITS, 2>(a, grid, team, part, cut, s);
}

}  // namespace

// Few items of short contexts: a cluster of CTAs per item, which join their parts through shared memory, without
// the line's scan and a second launch.  Long contexts and many items: the line, whose shares are even.  Contexts of
// a few units: an item per CTA.
int step_grid(const Args& a, int* team) {
  const int64_t units = ((a.table_width << a.page_shift) + ST_UNIT - 1) / ST_UNIT;
  const int64_t items = static_cast<int64_t>(a.seqs) * a.kv_heads;
  const int64_t slots = static_cast<int64_t>(eight(a) ? 3 : 2) * num_sms();
  *team = units <= 8 ? 1 : 0;
  if (units > 2 && units <= 64)
    for (int x = 2; x <= 8; x *= 2)
      if (items * x <= slots && x <= units) *team = x;
  if (*team == 0) return static_cast<int>(std::min(items * units, slots));
  return static_cast<int>(std::min<int64_t>(items, 1 << 20)) * *team;
}

int run_step(const Args& a, int dtype, int head_dim, int bits, int grid, int team, float* part, Cut* cut,
             cudaStream_t s) {
#define GPTQ_STEP(T, D)                                                                                        \
  return bits == 16  ? run<T, D, 16>(a, grid, team, part, cut, s)                                               \
         : bits == 8 ? run<T, D, 8>(a, grid, team, part, cut, s)                                                \
                     : run<T, D, 4>(a, grid, team, part, cut, s)
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
