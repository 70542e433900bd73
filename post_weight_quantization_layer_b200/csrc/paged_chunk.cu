// Attention over a paged cache for sequences with many rows (chunks of a prompt), on the tcgen05
// tensor cores.
//
// A tile is 256 rows of one kv head (row i * group + g of a sequence, so that all query heads of the kv
// head share its keys), two halves of 128 rows with a warpgroup each.  Per 128 keys and half: scores
// S = Q K^T into tensor memory, softmax by one thread per row, probabilities back into tensor memory
// over the scores, O += P V from there.  While one half's softmax runs, the tensor core works on the
// other half.  512 columns of tensor memory: two S (128 each, P over them), two O (head_dim each).
//
//  * Roles: warps 0-3 and 4-7 softmax, rescaling and output of their half; warp 8 issues the matrix
//    products; warp 9 walks the CTA's share, tells the others of each piece and brings keys and values; warps 10
//    and 11 bring the queries of a half as soon as its last scores are done; warps 12-19 (8- and 4-bit caches
//    only) turn codes into 16-bit operands.  Registers move to the softmax.
//  * 16-bit pages come by TMA straight into the swizzled operand tiles.  Pages of codes come by bulk
//    copies (codes, scales and zeros of a page and head are contiguous) into a staging ring, from
//    which the converters write operand tiles.  Keys are multiplied as code - zero, at most 8 bits and a sign and
//    so exact in q's type, and their scales multiply the scores in fp32; values as (code - zero) times their scale's
//    power of two, exact too, and the rest of the scale multiplies the probabilities in fp32, before they are rounded.
//    So nothing behind a code is rounded, nor a query, whatever its size; what remains is the rounding of the weights,
//    as over a 16-bit cache.  (All multiplied out and rounded, keys and bfloat16 queries to float16, values to q's type,
//    a long cache of 8 bits took 11 % less time: scores were -infinity, unnoticed, where 65504 was exceeded, and errors
//    1.7 times those of an answer in fp32 rounded once, now 1.41.)  A float16 call's value past that type's range is
//    infinite, makes its rows infinite or NaN, and is found by the second look.
//  * The running maximum moves only when it grows by more than 8 (base 2): until then weights reach 2^8 times what
//    they are held against, harmless in fp32 sums and 16-bit operands, and the accumulator needs no rescaling.
//  * The (row tile, 128 keys) units of the batch are cut into equal shares, one per SM, as in the
//    kernel for few rows; cut tiles are joined by a second launch in a fixed order.
// Bound by the exponentials and the tensor core together: 128 x 128 scores take 512 cycles of the
// tensor core twice and 1024 cycles of the 16-per-cycle exponential unit.  A half's turn takes about 2000 cycles
// of softmax and 850 of waiting for its products, and two halves share the tensor core: 1.15-1.24 PFLOP/s over a
// long 16-bit cache (1024 new tokens, 64 heads over 8, 16384 keys: 436 us; the clock falls to 1.4 GHz).
// Codes cost the converters' instructions, the scales' in the softmax and shared-memory traffic beside the tensor
// core's own: 721 us in 8 bits among calls with other inputs (691 from a graph that replays one), 742 (736) in 4.  Short
// prompts pay for each tile's start and end, about 9500 of 37000 cycles (four of 2048, 32 heads: 219 us, 187 from a
// graph).
#include <cuda.h>

#include <algorithm>
#include <mutex>

#include "paged.cuh"
#include "paged_plan.cuh"
#include "sm100.cuh"

namespace gptq {
namespace paged {
namespace {

using namespace sm100;

constexpr int CH_ROWS = kTileRows;
constexpr int CH_KEYS = 128;  // keys of a unit
constexpr int CH_RAW = 64;    // keys of a staging slot
constexpr uint32_t CH_WAIT = 1u << 22;
constexpr float CH_GROW = 8.f;  // an online softmax that rescales only where the maximum grew by more (base 2)

__device__ int g_chunk_status = 0;

template <int D, int BITS>
struct Cfg {
  static constexpr int CONV = BITS == 16 ? 0 : 256;     // converting threads
  static constexpr int THREADS = 384 + CONV;
  static constexpr int TILE = CH_KEYS * D * 2;         // bytes of an operand tile
  static constexpr int NST = D == 128 ? 4 : 6;         // operand tiles in the ring
  static constexpr int ROW = D * BITS / 8;
  // staging of codes and zeros, half a tile of keys or values each
  static constexpr int RAW = BITS == 16 ? 0 : CH_RAW * (ROW + 1);
  static constexpr int NRAW = BITS == 16 ? 1 : 4;      // two halves of keys, two of values
  // places for the scales of a tile's keys and values: as many as the ring has for operands of values (one more, and no
  // wait for a free one, has no room beside 8-bit keys of 128 and gained nothing elsewhere)
  static constexpr int NSC = BITS == 16 ? 0 : NST / 2;
  static constexpr int QOFF = 0;
  static constexpr int RING = 2 * TILE;
  static constexpr int ROFF = RING + NST * TILE;
  static constexpr int SCALES = ROFF + NRAW * RAW;
  static constexpr int BARS = SCALES + NSC * 2 * CH_KEYS * 4;
  static constexpr int NBARS = 2 * NST + 2 * NRAW + 2 * NSC + 18;
  static constexpr int JOBS = BARS + NBARS * 8 + 8;
  static constexpr int SMEM = JOBS + 2 * 40;
  static_assert(SMEM <= 232448, "shared memory of a CTA");
  static_assert(RAW % 16 == 0, "bulk copies start on 16 bytes");
};

// ------------------------------------------------------------------ the line of units
struct Tile {
  int kend;   // keys that the tile's last row sees
  int units;  // of CH_KEYS keys; 1 where there is none
};

__device__ __forceinline__ Tile tile_of(const Args& a, const Seq& q, int tile) {
  Tile t;
  const int last = min(q.n - 1, static_cast<int>((static_cast<uint32_t>(tile + 1) * CH_ROWS - 1) / static_cast<uint32_t>(a.group)));
  t.kend = seen(a, q, last);
  t.units = max(1, (t.kend + CH_KEYS - 1) / CH_KEYS);
  return t;
}

__device__ __forceinline__ int tiles_of(const Args& a, const Seq& q) {
  const int64_t rows = static_cast<int64_t>(q.n) * a.group;
  return rows > kStepRows ? static_cast<int>((rows + CH_ROWS - 1) / CH_ROWS) : 0;
}

__device__ int64_t head_units(const Args& a, int s) {  // units of one kv head of sequence s
  const Seq q = sequence(a, s);
  const int n = tiles_of(a, q);
  int64_t u = 0;
  for (int i = 0; i < n; ++i) u += tile_of(a, q, i).units;
  return u;
}

struct Piece {
  int64_t at, end;
  int s, head, tile, u0, u1, units, tiles, kend;
  Seq q;
};

__device__ __forceinline__ void enter_tile(const Args& a, Piece& p, int u0) {
  const Tile t = tile_of(a, p.q, p.tile);
  p.kend = t.kend;
  p.units = t.units;
  p.u0 = u0;
  p.u1 = static_cast<int>(min(static_cast<int64_t>(t.units), u0 + (p.end - p.at)));
}

// The first piece of share `cta`; false where it is empty.  All threads; shared: 3 + THREADS / 32 * 9 words.
template <int THREADS>
__device__ bool chunk_first(const Args& a, int64_t cta, Piece& p, int64_t& per, int64_t* shared) {
  int64_t all = 0, total;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  constexpr int WARPS = THREADS / 32;
  int64_t* sums = shared + 3 + WARPS;
  const bool few = a.seqs <= 8 * WARPS;  // a warp per sequence, a lane per tile; otherwise a thread per sequence
  if (few) {
    for (int x = warp; x < a.seqs; x += WARPS) {
      const Seq q = sequence(a, x);
      const int n = tiles_of(a, q);
      int64_t u = 0;
      for (int i = lane; i < n; i += 32) u += tile_of(a, q, i).units;
      for (int o = 16; o; o >>= 1) u += __shfl_xor_sync(0xffffffffu, u, o);
      if (lane == 0) sums[x] = u;
    }
    __syncthreads();
    if (threadIdx.x < a.seqs) all = sums[threadIdx.x];
  } else {
    for (int x = threadIdx.x; x < a.seqs; x += THREADS) all += head_units(a, x);
  }
  const int64_t upto = block_scan<THREADS>(all, total, shared + 3) * a.kv_heads;
  total *= a.kv_heads;
  // Few units: a CTA each, since a unit takes longer than its part takes to join (206 tokens of 64 heads over 281
  // keys: 28 us instead of 43 with 8 units at least and 30 with 4; 64 tokens alone: 20, 60 and 37).
  per = (total + gridDim.x - 1) / gridDim.x;
  p.at = cta * per;
  p.end = min(total, p.at + per);
  if (p.at >= p.end) return false;
  auto take = [&](int x, int64_t u, int64_t lo) {
    if (u && lo <= p.at && p.at < lo + u) {
      shared[0] = x;
      shared[1] = p.at - lo;
      shared[2] = u / a.kv_heads;
    }
  };
  if (a.seqs <= THREADS) {
    take(threadIdx.x, all * a.kv_heads, upto - all * a.kv_heads);
  } else {
    int64_t base = 0;
    for (int x0 = 0; x0 < a.seqs; x0 += THREADS) {
      const int x = x0 + threadIdx.x;
      const int64_t u = x < a.seqs ? head_units(a, x) * a.kv_heads : 0;
      int64_t sum;
      const int64_t incl = block_scan<THREADS>(u, sum, shared + 3);
      take(x, u, base + incl - u);
      base += sum;
      if (base > p.at) break;
    }
  }
  __syncthreads();
  p.s = static_cast<int>(shared[0]);
  p.q = sequence(a, p.s);
  p.tiles = tiles_of(a, p.q);
  p.head = static_cast<int>(shared[1] / shared[2]);
  int64_t rem = shared[1] % shared[2];
  // the tile that holds unit `rem` of the head: every warp finds it, 32 tiles at a time
  for (p.tile = 0;; p.tile += 32) {
    const int mine = p.tile + lane < p.tiles ? tile_of(a, p.q, p.tile + lane).units : 0;
    int upto32 = mine;
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, upto32, o);
      if (lane >= o) upto32 += x;
    }
    const unsigned past = __ballot_sync(0xffffffffu, rem < upto32);
    if (past) {
      const int l = __ffs(past) - 1;
      p.tile += l;
      rem -= __shfl_sync(0xffffffffu, upto32 - mine, l);
      break;
    }
    if (p.tile + 32 >= p.tiles) break;  // (does not happen: the head's units are the tiles')
    rem -= __shfl_sync(0xffffffffu, upto32, 31);
  }
  enter_tile(a, p, static_cast<int>(rem));
  return true;
}

__device__ __forceinline__ void chunk_next(const Args& a, Piece& p) {
  p.at += p.u1 - p.u0;
  if (p.at >= p.end) return;
  if (++p.tile == p.tiles) {
    p.tile = 0;
    if (++p.head == a.kv_heads) {
      p.head = 0;
      do {
        ++p.s;
        p.q = sequence(a, p.s);
        p.tiles = tiles_of(a, p.q);
      } while (p.tiles == 0);
    }
  }
  enter_tile(a, p, 0);
}

// ------------------------------------------------------------------ instructions
// Shared-memory descriptors as their low word (start address and leading offset, 16-byte units: a step
// inside a tile is an addition) with a constant high word (stride 1024 bytes, version 1, 128-byte swizzle).
constexpr uint32_t DESC_HI = (1024u >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ constexpr uint32_t desc_lo(uint32_t saddr, uint32_t lbo) { return (saddr >> 4) | ((lbo >> 4) << 16); }

// D[tmem] (+)= A[smem] * B[smem], kind::f16.
__device__ __forceinline__ void umma_ss(uint32_t tmem_d, uint32_t alo, uint32_t blo, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "mov.b64 a, {%1, %5};\n\t"
      "mov.b64 b, {%2, %5};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p;\n\t}" ::"r"(tmem_d),
      "r"(alo), "r"(blo), "r"(idesc), "r"(accumulate), "r"(DESC_HI)
      : "memory");
}
// D[tmem] (+)= A[tmem] * B[smem], kind::f16.
__device__ __forceinline__ void umma_ts(uint32_t tmem_d, uint32_t tmem_a, uint32_t blo, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 b;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "mov.b64 b, {%2, %5};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %3, p;\n\t}" ::"r"(tmem_d),
      "r"(tmem_a), "r"(blo), "r"(idesc), "r"(accumulate), "r"(DESC_HI)
      : "memory");
}

// Loads without their wait: the registers may be used after tmem_ld_wait() and settled().
__device__ __forceinline__ void tmem_ld_x32_nowait(uint32_t taddr, float (&v)[32]) {
  uint32_t* r = reinterpret_cast<uint32_t*>(v);
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
        "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]),
        "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]),
        "=r"(r[30]), "=r"(r[31])
      : "r"(taddr)
      : "memory");
}
// Orders uses of the registers after the wait that precedes it.
__device__ __forceinline__ void settled(float (&v)[32]) {
#pragma unroll
  for (int i = 0; i < 32; i += 8)
    asm volatile("" : "+f"(v[i]), "+f"(v[i + 1]), "+f"(v[i + 2]), "+f"(v[i + 3]), "+f"(v[i + 4]), "+f"(v[i + 5]),
                      "+f"(v[i + 6]), "+f"(v[i + 7]));
}
__device__ __forceinline__ void tmem_ld_x16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_st_x16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};" ::"r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
      "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
}

__device__ __forceinline__ void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// Untiled copy global -> shared (16-byte aligned, a multiple of 16 bytes).
__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                   smem_u32(dst)),
               "l"(src), "r"(bytes), "r"(smem_u32(bar))
               : "memory");
}

template <int N>
__device__ __forceinline__ void regs_more() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_fewer() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
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
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
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

__device__ __forceinline__ void store32(void* p, const uint32_t* v) {
  asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]),
               "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}

// A value's scale is a power of two with the sign, by which its codes are multiplied, exactly, times a part of 1 .. 2, by
// which its weight is.  (Below float32's normal range: the scale, and 1.)
__device__ __forceinline__ float power_of(float s) {
  const uint32_t w = __float_as_uint(s);
  return (w & 0x7f800000u) ? __uint_as_float(w & 0xff800000u) : s;
}
__device__ __forceinline__ float part_of(float s) {
  const uint32_t w = __float_as_uint(s);
  return (w & 0x7f800000u) ? __uint_as_float((w & 0x007fffffu) | 0x3f800000u) : 1.f;
}

// Scores of 32 keys times their scales, which are taken before the wait for the scores.
__device__ __forceinline__ void take_scales(float4 (&s)[8], const float* scales) {
#pragma unroll
  for (int e = 0; e < 8; ++e) s[e] = *reinterpret_cast<const float4*>(scales + 4 * e);
}
__device__ __forceinline__ void by_scales(float (&x)[32], const float4 (&s)[8]) {
#pragma unroll
  for (int e = 0; e < 32; e += 4) {
    const float2 lo = mul2(make_float2(x[e], x[e + 1]), make_float2(s[e / 4].x, s[e / 4].y));
    const float2 hi = mul2(make_float2(x[e + 2], x[e + 3]), make_float2(s[e / 4].z, s[e / 4].w));
    x[e] = lo.x;
    x[e + 1] = lo.y;
    x[e + 2] = hi.x;
    x[e + 3] = hi.y;
  }
}

// Scores of keys (from `key`) that the row does not see become -infinity.
__device__ __forceinline__ void hide(float (&x)[32], int key, int see) {
#pragma unroll
  for (int e = 0; e < 32; ++e) x[e] = key + e < see ? x[e] : -INFINITY;
}

template <int N>
__device__ __forceinline__ float highest(const float (&x)[N][32]) {
  float m[8];
#pragma unroll
  for (int c = 0; c < 8; ++c) m[c] = fmaxf(x[0][c], x[0][c + 8]);
#pragma unroll
  for (int y = 16; y < N * 32; y += 16)
#pragma unroll
    for (int c = 0; c < 8; ++c) m[c] = max3(m[c], x[y >> 5][(y & 31) + c], x[y >> 5][(y & 31) + c + 8]);
  return max3(max3(m[0], m[1], m[2]), max3(m[3], m[4], m[5]), fmaxf(m[6], m[7]));
}

// Probabilities 2^(score scale + ref) of a row's 128 scores into tensor memory as 16-bit pairs, over the
// scores: part c of 32 keys takes columns that part c / 2 has left.  x holds the first parts, the others are
// read again (and, over codes, multiplied by their keys' scales again).  Returns the sum; arrives at `most` and
// `full` as they get there.  All go through the exponential unit: a share of them by polynomial was faster alone
// (959 cycles instead of 1168 for a warp with three of eight) and slower here (prompts of 2048, 32 heads: 244 us
// instead of 223), where its registers and issue slots are missed.
template <typename T, int BITS, int KEEP>
__device__ __forceinline__ float weights(float (&x)[KEEP][32], const float* scales, float scale, float ref, uint32_t dst,
                                         int key, int see, int least, uint64_t* most, uint64_t* full) {
  const float* parts = scales + CH_KEYS;  // of the values' scales
  const float2 sc2 = make_float2(scale, scale), ref2 = make_float2(ref, ref);
  float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    float(&v)[32] = x[c % KEEP];
    if (c >= KEEP) {
      float4 s[8];
      if constexpr (BITS < 16) take_scales(s, scales + c * 32);
      tmem_ld_wait();
      settled(v);
      if constexpr (BITS < 16) by_scales(v, s);
      if (key + CH_KEYS > least) hide(v, key + c * 32, see);
    }
    uint32_t r[16];
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      float2 p = fma2(make_float2(v[2 * e], v[2 * e + 1]), sc2, ref2);
      p.x = ex2(p.x);
      p.y = ex2(p.y);
      sum[e & 1] = add2(sum[e & 1], p);
      if constexpr (BITS < 16) p = mul2(p, *reinterpret_cast<const float2*>(parts + c * 32 + 2 * e));
      r[e] = pack2<T>(p.x, p.y);
    }
    if (c + KEEP < 4) tmem_ld_x32_nowait(dst + (c + KEEP) * 32, v);
    tmem_st_x16(dst + c * 16, r);
    if (c >= 2) {  // the first 96 keys may be multiplied while the last are on their way
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if ((threadIdx.x & 31) == 0) mbar_arrive(c == 2 ? most : full);
    }
  }
  return (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
}

// Byte offset of 16-byte chunk c (8 elements) of row r in an operand tile: 64-element blocks of [128 rows]
// [128 bytes], 128-byte swizzle.
__device__ __forceinline__ uint32_t chunk_off(int r, int c) {
  return static_cast<uint32_t>((c >> 3) * (CH_KEYS * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4));
}

struct Bars {
  uint64_t *full, *empty, *rfull, *rempty, *scales, *parts, *jfull, *jempty, *qfull, *qfree, *sfull, *pmost, *pfull;
  uint64_t *odone, *zero, *done;
};

// What the other warps have to know of a piece, as the warp that walks the line tells them through shared
// memory (two entries in turn): they then keep little of it in registers.
struct Job {
  int start, n, len;  // the sequence
  int head, tile;
  int key0, kend;     // keys of the piece
  int tiles;          // of CH_KEYS keys; -1: no piece is left
  int tiles0;         // of which the first half's rows see some key
  int slot;           // where the part is left behind: 0 or 1 of the CTA; -1: the tile is whole
};
static_assert(sizeof(Job) == 40, "Job");

// A reader's side of the jobs: waits for the next one, takes a copy and gives the entry back.
struct JobReader {
  const Job* jobs;
  uint64_t *full, *empty;
  int i = 0;
  uint32_t ph = 0;
  __device__ __forceinline__ JobReader(const Job* j, const Bars& b) : jobs(j), full(b.jfull), empty(b.jempty) {}
  // false where the wait ran out (job.tiles is then -1)
  __device__ __forceinline__ bool next(Job& job) {
    const bool there = mbar_wait(&full[i], ph, CH_WAIT);
    if (there)
      job = jobs[i];
    else
      job.tiles = -1;
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(&empty[i]);
    if (++i == 2) {
      i = 0;
      ph ^= 1u;
    }
    return there;
  }
};

// A place in a ring of N: index and phase.
template <int N>
struct Ring {
  int i = 0;
  uint32_t ph = 0;
  __device__ __forceinline__ void step() {
    if (++i == N) {
      i = 0;
      ph ^= 1u;
    }
  }
};

template <typename T, int D, int BITS>
__global__ void __launch_bounds__(Cfg<D, BITS>::THREADS, 1)
    chunk_kernel(const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tv, const Args a,
                 float* __restrict__ part, Cut* __restrict__ cut, int* __restrict__ odd) {
  using C = Cfg<D, BITS>;
  constexpr int SIZE = chunk_part(D);
  constexpr int KEEP = BITS == 16 ? 4 : 2;
  constexpr uint32_t FMT = std::is_same<T, __half>::value ? 0u : 1u;
  // Of the keys' operands over codes, (code - zero) KEY_STEP: no product of a finite bfloat16 query and a key, and no
  // sum of them, is past fp32 then.
  constexpr float KEY_STEP = FMT ? 0x1p-16f : 1.f;
  // Weights in float16 are held against 2^7 (with CH_GROW, up to 2^15): many keys that weigh under 2^-25 of the
  // largest, float16's last step, may count for something together.
  constexpr float UP = FMT ? 0.f : (BITS == 16 ? 7.f : 6.f);  // (over codes they are up to twice as large)
  extern __shared__ __align__(1024) uint8_t smem[];  // the swizzle's unit
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  next_may_start();
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::BARS);
  Bars b;
  b.full = bars;
  b.empty = b.full + C::NST;
  b.rfull = b.empty + C::NST;
  b.rempty = b.rfull + C::NRAW;
  b.scales = b.rempty + C::NRAW;
  b.parts = b.scales + C::NSC;
  b.jfull = b.parts + C::NSC;
  b.jempty = b.jfull + 2;
  b.qfull = b.jempty + 2;
  b.qfree = b.qfull + 2;
  b.sfull = b.qfree + 2;
  b.pmost = b.sfull + 2;
  b.pfull = b.pmost + 2;
  b.odone = b.pfull + 2;
  b.zero = b.odone + 2;
  b.done = b.zero + 1;
  uint32_t* slot = reinterpret_cast<uint32_t*>(b.done + 1);
  int* any_odd = reinterpret_cast<int*>(slot + 1);
  Job* jobs = reinterpret_cast<Job*>(smem + C::JOBS);
  if (threadIdx.x == 0) {
    for (int i = 0; i < C::NST; ++i) {
      mbar_init(&b.full[i], BITS == 16 ? 1 : 4);
      mbar_init(&b.empty[i], 1);
    }
    for (int i = 0; i < C::NRAW; ++i) {
      mbar_init(&b.rfull[i], 1);
      mbar_init(&b.rempty[i], 4);
    }
    for (int i = 0; i < C::NSC; ++i) {
      mbar_init(&b.scales[i], 1);
      mbar_init(&b.parts[i], 4);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&b.jfull[i], 1);
      mbar_init(&b.jempty[i], 11 + C::CONV / 32);  // softmax, issuing, query and converting warps
      mbar_init(&b.qfull[i], 1);
      mbar_init(&b.qfree[i], 1);
      mbar_init(&b.sfull[i], 1);
      mbar_init(&b.pmost[i], 4);
      mbar_init(&b.pfull[i], 4);
      mbar_init(&b.odone[i], 1);
    }
    *any_odd = 0;
    mbar_init(b.zero, 1);
    mbar_init(b.done, 1);
    fence_barrier_init();
  }
  if (warp == 8) {
    tmem_alloc(slot, 512);
    tmem_relinquish();
  }
  Piece p;
  int64_t per;
  // (the operand ring is not in use yet)
  const bool any = chunk_first<C::THREADS>(a, blockIdx.x, p, per, reinterpret_cast<int64_t*>(smem));
  if (threadIdx.x == 0) {
    cut[blockIdx.x] = any ? cut_at(p.at, per, p.u0, p.units, p.q, p.head, p.tile) : Cut{0, -1};
    if (!any) odd[blockIdx.x] = 0;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (!any) {
    if (warp == 8) tmem_dealloc(*slot, 512);
    wait_for_last();
    return;
  }
  const int64_t first = p.at;

  const uint32_t tmem = *slot;
  bool ok = true;

  if (warp < 8) {
    // ---------------------------------------------------------------- softmax, one thread per row
    regs_more<BITS == 16 ? 216 : 136>();
    const int w = warp >> 2, wr = (warp & 3) * 32 + lane;  // half, row of the half
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t S = tmem + lanes + w * 128, O = tmem + lanes + 256 + w * D;
    uint32_t sph = 0, oph = 0;
    const bool wide = (reinterpret_cast<uintptr_t>(a.out) & 31u) == 0;
    JobReader reader(jobs, b);
    Job job;
    const float scale = BITS < 16 ? a.scale_log2 * (1.f / KEY_STEP) : a.scale_log2;
    uint32_t before = 0, told = 0;  // tiles of the pieces before this one, and with it: the place of their scales
    auto next_job = [&]() {  // the next piece whose tile has this half
      do {
        if (!reader.next(job)) ok = false;
        before = told;
        told += max(job.tiles, 0);
      } while (job.tiles >= 0 && job.tile * CH_ROWS + w * 128 >= job.n * a.group);
      return job.tiles >= 0;
    };
    while (next_job()) {
      const int row = job.tile * CH_ROWS + w * 128 + wr;
      const bool in = row < job.n * a.group;
      const int i = in ? static_cast<uint32_t>(row) / static_cast<uint32_t>(a.group) : 0;
      const int h = job.head * a.group + (in ? row - i * a.group : 0);
      const int tiles = w ? job.tiles : job.tiles0;
      int key = job.key0;
      const Seq q{job.start, job.n, job.len};
      const int see = in ? min(job.kend, seen(a, q, i)) : job.kend;  // rows past the last: what comes out is not used
      int least = see;
      for (int o = 16; o; o >>= 1) least = min(least, __shfl_xor_sync(0xffffffffu, least, o));
      float* mine = job.slot < 0 ? nullptr
                                 : part + (static_cast<int64_t>(blockIdx.x) * 2 + job.slot) * static_cast<int64_t>(SIZE) +
                                       w * 128 + wr;
      T* dst = static_cast<T*>(a.out) + ((static_cast<int64_t>(job.start) + i) * a.heads + h) * D;
      float m = -INFINITY, l = 0.f;
      for (int j = 0; j < tiles; ++j, key += CH_KEYS) {
        if (!mbar_wait(&b.sfull[w], sph, CH_WAIT)) {
          ok = false;
          break;
        }
        sph ^= 1u;
        const float* scales = nullptr;
        if constexpr (BITS < 16) {
          // (the scores are there, so the scales of all earlier tiles have come)
          const uint32_t at = before + j, turn = at / C::NSC, place = at - turn * C::NSC;
          if (!mbar_wait(&b.scales[place], turn & 1u, CH_WAIT) || !mbar_wait(&b.parts[place], turn & 1u, CH_WAIT)) {
            ok = false;
            break;
          }
          scales = reinterpret_cast<const float*>(smem + C::SCALES) + place * 2 * CH_KEYS;
        }
        __syncwarp();  // tensor memory is read by whole warps, and a wait ends thread by thread
        tc_fence_after();
        // The maximum first, then the probabilities: only KEEP of the four 32-key parts of the scores stay in
        // registers between the two, the others are read from tensor memory again.
        float x[KEEP][32];
        float top = -INFINITY;
        // (Two turns of one loop over codes: unrolled as well, the converters and the softmax miss the instruction
        // cache more, by 3 % over a long chunk of 8 bits and 8 % in prompts.)
#pragma unroll 1
        for (int c = 4 - KEEP; c >= 0; c -= KEEP) {
#pragma unroll
          for (int y = 0; y < KEEP; ++y) tmem_ld_x32_nowait(S + (c + y) * 32, x[y]);
          float4 s[8];
          if constexpr (BITS < 16) take_scales(s, scales + c * 32);
          tmem_ld_wait();
#pragma unroll
          for (int y = 0; y < KEEP; ++y) {
            settled(x[y]);
            if constexpr (BITS < 16) {
              if (y) take_scales(s, scales + (c + y) * 32);
              by_scales(x[y], s);
            }
          }
          if (key + CH_KEYS > least) {
#pragma unroll
            for (int y = 0; y < KEEP; ++y) hide(x[y], key + (c + y) * 32, see);
          }
          top = fmaxf(top, highest(x));
        }
        if (j == 0) {
          m = top;
        } else if (__any_sync(0xffffffffu, (top - m) * scale > CH_GROW)) {
          // all earlier products are complete: they precede these scores on the tensor core
          const float now = fmaxf(m, top);
          const float f = now == -INFINITY ? 1.f : ex2((m - now) * scale);
          m = now;
          l *= f;
#pragma unroll
          for (int c = 0; c < D / 16; ++c) {
            uint32_t r[16];
            tmem_ld_x16(O + c * 16, r);
#pragma unroll
            for (int e = 0; e < 16; ++e) r[e] = __float_as_uint(__uint_as_float(r[e]) * f);
            tmem_st_x16(O + c * 16, r);
          }
        }
        const float ref = m == -INFINITY ? 0.f : UP - m * scale;
        l += weights<T, BITS, KEEP>(x, scales, scale, ref, S, key, see, least, &b.pmost[w], &b.pfull[w]);
      }
      if (!ok) break;
      if (tiles) {
        if (!mbar_wait(&b.odone[w], oph, CH_WAIT)) {
          ok = false;
          break;
        }
        oph ^= 1u;
        __syncwarp();
        tc_fence_after();
      }
      const float inv = l == 0.f ? 0.f : 1.f / l;
      float2 odd2 = make_float2(0.f, 0.f);  // NaN as soon as one value is not finite
#pragma unroll
      for (int c = 0; c < D / 32; ++c) {
        float o[32];
        if (tiles) {
          tmem_ld_32x32b_x32(O + c * 32, o);
        } else {
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = 0.f;
        }
#pragma unroll
        for (int e = 0; e < 32; e += 2) odd2 = fma2(make_float2(o[e], o[e + 1]), make_float2(0.f, 0.f), odd2);
        if (mine) {
#pragma unroll
          for (int e = 0; e < 32; ++e) mine[(c * 32 + e) * CH_ROWS] = o[e];
          continue;
        }
        uint32_t v[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) v[e] = pack2<T>(o[2 * e] * inv, o[2 * e + 1] * inv);
        if (in) {
          // a row per lane: the wider the stores, the fewer lines they touch
          if (wide) {
            store32(dst + c * 32, v);
            store32(dst + c * 32 + 16, v + 8);
          } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
              reinterpret_cast<uint4*>(dst)[c * 4 + e] = make_uint4(v[4 * e], v[4 * e + 1], v[4 * e + 2], v[4 * e + 3]);
          }
        }
      }
      const bool fine = odd2.x + odd2.y == 0.f;
      if (mine) {
        mine[D * CH_ROWS] = m == -INFINITY ? m : m * scale - UP;
        mine[(D + 1) * CH_ROWS] = l;
      }
      tc_fence_before();
      if (in && !fine) *any_odd = 1;
    }
  } else if (warp < 12) {
    regs_fewer<72>();
    if (warp == 8) {
      // -------------------------------------------------------------- issue of the matrix products
      // The whole warp walks the loops and one elected lane issues: descriptors then stay in uniform
      // registers (a product issues every 66 cycles; from a single lane's branch every 82, measured alone).
      constexpr uint32_t iqk = instr_desc(FMT, false, false, 128, CH_KEYS);
      constexpr uint32_t ipv = instr_desc(FMT, false, true, 128, D);
      const bool lead = elect_one();
      Ring<C::NST> ring;
      uint32_t qph = 0, pph = 0;  // phases, a bit per half
      const uint32_t q0 = desc_lo(smem_u32(smem + C::QOFF), 16), k0 = desc_lo(smem_u32(smem + C::RING), 16);
      const uint32_t v0 = desc_lo(smem_u32(smem + C::RING), CH_KEYS * 128);
      auto qk = [&](int w, int st, bool last) {
        const uint32_t qa = q0 + w * (C::TILE >> 4), kb = k0 + st * (C::TILE >> 4);
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          const uint32_t off = static_cast<uint32_t>((k >> 2) * (CH_KEYS * 128) + (k & 3) * 32) >> 4;
          umma_ss(tmem + w * 128, qa + off, kb + off, iqk, k > 0 ? 1u : 0u);
        }
        umma_commit(&b.sfull[w]);
        if (last) umma_commit(&b.qfree[w]);  // the piece's last scores: its queries are done with
      };
      JobReader reader(jobs, b);
      Job job;
      while (ok) {
        ok = reader.next(job);
        if (job.tiles < 0) break;
        const bool two = job.n * a.group > job.tile * CH_ROWS + 128;  // the tile has a second half
        // tiles of each half: the second half's rows see at least as many keys
        const int n0 = job.tiles0, n1 = two ? job.tiles : 0, tiles = max(n0, n1);
        if (tiles) ok = mbar_wait(&b.full[ring.i], ring.ph, CH_WAIT);
        if (!ok) break;
#pragma unroll
        for (int w = 0; w < 2; ++w) {
          if ((w ? n1 : n0) == 0) continue;
          ok = ok && mbar_wait(&b.qfull[w], (qph >> w) & 1u, CH_WAIT);  // Q of this piece is in place
          qph ^= 1u << w;
          tc_fence_after();
          if (ok && lead) qk(w, ring.i, (w ? n1 : n0) == 1);
          __syncwarp();
        }
        if (!ok) break;
        if (!tiles) continue;
        if (lead) umma_commit(&b.empty[ring.i]);
        __syncwarp();
        ring.step();
        for (int j = 0; j < tiles && ok; ++j) {
          const int vst = ring.i;
          const uint32_t vph = ring.ph;
          ring.step();
          const int kst = ring.i;
          const uint32_t kph = ring.ph;
          const bool more = j + 1 < tiles;
          if (more) ring.step();
          ok = ok && mbar_wait(&b.full[vst], vph, CH_WAIT);
          if (more) ok = ok && mbar_wait(&b.full[kst], kph, CH_WAIT);
#pragma unroll
          for (int w = 0; w < 2; ++w) {
            const int mine = w ? n1 : n0;
            if (j >= mine) continue;
            const uint32_t vb = v0 + vst * (C::TILE >> 4);
            ok = ok && mbar_wait(&b.pmost[w], (pph >> w) & 1u, CH_WAIT);
            if (!ok) break;
            tc_fence_after();
            if (lead) {
#pragma unroll
              for (int k = 0; k < 6; ++k)
                umma_ts(tmem + 256 + w * D, tmem + w * 128 + k * 8, vb + k * (2048 >> 4), ipv, (j > 0 || k > 0) ? 1u : 0u);
            }
            __syncwarp();
            ok = mbar_wait(&b.pfull[w], (pph >> w) & 1u, CH_WAIT);
            pph ^= 1u << w;
            if (!ok) break;
            tc_fence_after();
            if (lead) {
#pragma unroll
              for (int k = 6; k < CH_KEYS / 16; ++k)
                umma_ts(tmem + 256 + w * D, tmem + w * 128 + k * 8, vb + k * (2048 >> 4), ipv, 1u);
              if (w == 1 || n1 <= j) umma_commit(&b.empty[vst]);  // no half after this one uses the values
              if (j + 1 < mine)
                qk(w, kst, j + 2 == mine);
              else
                umma_commit(&b.odone[w]);
              if (more && (w == 1 || n1 <= j)) umma_commit(&b.empty[kst]);
            }
            __syncwarp();
          }
        }
      }
      if (lead) umma_commit(b.done);
      __syncwarp();
      mbar_wait(b.done, 0, CH_WAIT);
    } else if (warp == 9) {
      // -------------------------------------------------------------- keys and values, page by page
      Ring<C::NST> ring;
      Ring<C::NRAW> raw;
      uint32_t zph = 0;
      int issued = 0;
      const int box = min(1 << a.page_shift, BITS == 16 ? CH_KEYS : CH_RAW), boxes = CH_KEYS / box;
      int ji = 0;
      uint32_t jph = 1u;
      // The scales of a tile's keys and values come with the first half of its values, when the place of these values'
      // operands is free: the softmax is past the tile that had it, and so past the last user of the scales' place.
      Ring<C::NSC ? C::NSC : 1> keyed;
      int scaled = 0;
      auto tell = [&](const Job& job) {
        if (!mbar_wait(&b.jempty[ji], jph, CH_WAIT)) return false;
        if (lane == 0) {
          jobs[ji] = job;
          mbar_arrive(&b.jfull[ji]);
        }
        __syncwarp();
        if (++ji == 2) {
          ji = 0;
          jph ^= 1u;
        }
        return true;
      };
      for (; p.at < p.end && ok; chunk_next(a, p)) {
        const int tiles = p.kend > 0 ? p.u1 - p.u0 : 0;
        const bool whole = p.u0 == 0 && p.u1 == p.units;
        const uint32_t mid = (static_cast<uint32_t>(p.tile) * CH_ROWS + 127) / static_cast<uint32_t>(a.group);
        const int kend0 = seen(a, p.q, min(p.q.n - 1, static_cast<int>(mid)));
        const int tiles0 = max(0, min(tiles, (kend0 + CH_KEYS - 1) / CH_KEYS - p.u0));
        ok = tell(Job{p.q.start, p.q.n, p.q.len, p.head, p.tile, p.u0 * CH_KEYS, min(p.u1 * CH_KEYS, p.kend), tiles, tiles0,
                      whole ? -1 : (p.at == first ? 0 : 1)});
        // a lane per box; the page of the next tile's box is looked up one tile ahead
        auto find = [&](int key) { return key + lane * box < p.kend && lane < boxes ? key_at(a, p.s, p.head, key + lane * box) : 0; };
        int64_t next = tiles ? find(p.u0 * CH_KEYS) : 0;
        for (int j = 0; j < tiles && ok; ++j) {
          const int key = (p.u0 + j) * CH_KEYS;
          const int n = min(boxes, (p.kend - key + box - 1) / box);  // boxes that hold keys
          const int64_t at = next;
          if (j + 1 < tiles) next = find(key + CH_KEYS);
          for (int kv = 0; kv < 2; ++kv) {
            if constexpr (BITS == 16) {
              if (!mbar_wait(&b.empty[ring.i], ring.ph ^ 1u, CH_WAIT)) {
                ok = false;
                break;
              }
              uint8_t* dst = smem + C::RING + ring.i * C::TILE;
              // the last values of a sequence: what lies behind them in the tile must be finite
              const int rest = p.kend - key;
              const bool tail = kv == 1 && rest < CH_KEYS;
              uint64_t* bar = tail ? b.zero : &b.full[ring.i];
              if (lane == 0) mbar_arrive_expect_tx(bar, static_cast<uint32_t>(n * box * D * 2));
              __syncwarp();
              if (lane < n) {
#pragma unroll
                for (int c = 0; c < D / 64; ++c)
                  tma_load_2d(dst + c * (CH_KEYS * 128) + lane * box * 128, kv ? &tv : &tk, bar, c * 64, static_cast<int>(at));
              }
              if (tail) {
                if (!mbar_wait(b.zero, zph, CH_WAIT)) {
                  ok = false;
                  break;
                }
                zph ^= 1u;
                for (int e = lane; e < (CH_KEYS - rest) * (D / 8); e += 32) {
                  const int r = rest + e / (D / 8), c = e % (D / 8);
                  *reinterpret_cast<uint4*>(dst + chunk_off(r, c)) = make_uint4(0, 0, 0, 0);
                }
                fence_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&b.full[ring.i]);
              }
              ++issued;
              ring.step();
            } else {
              for (int hf = 0; hf < 2; ++hf) {
                if (!mbar_wait(&b.rempty[raw.i], raw.ph ^ 1u, CH_WAIT)) {
                  ok = false;
                  break;
                }
                if (kv == 1 && hf == 0) {
                  if (!mbar_wait(&b.empty[2 * keyed.i + 1], keyed.ph ^ 1u, CH_WAIT)) {
                    ok = false;
                    break;
                  }
                  if (lane == 0) mbar_arrive_expect_tx(&b.scales[keyed.i], static_cast<uint32_t>(n * box * 8));
                  __syncwarp();
                  if (lane < n) {
                    uint8_t* to = smem + C::SCALES + (keyed.i * 2 * CH_KEYS + lane * box) * 4;
                    bulk_load(to, a.ks + at, box * 4, &b.scales[keyed.i]);
                    bulk_load(to + CH_KEYS * 4, a.vs + at, box * 4, &b.scales[keyed.i]);
                  }
                  ++scaled;
                  keyed.step();
                }
                uint8_t* dst = smem + C::ROFF + raw.i * C::RAW;
                const int b0 = hf * (boxes / 2), nb = max(0, min(boxes / 2, n - b0));
                if (lane == 0) mbar_arrive_expect_tx(&b.rfull[raw.i], static_cast<uint32_t>(nb * box * (C::ROW + 1)));
                __syncwarp();
                if (lane >= b0 && lane < b0 + nb) {
                  const int x = (lane - b0) * box;
                  const uint8_t* codes = static_cast<const uint8_t*>(kv ? a.vc : a.kc) + at * C::ROW;
                  bulk_load(dst + x * C::ROW, codes, box * C::ROW, &b.rfull[raw.i]);
                  bulk_load(dst + CH_RAW * C::ROW + x, (kv ? a.vz : a.kz) + at, box, &b.rfull[raw.i]);
                }
                ++issued;
                raw.step();
              }
              if (!ok) break;
            }
          }
        }
      }
      if (ok) ok = tell(Job{0, 0, 0, 0, 0, 0, 0, -1, 0, 0});
      // no copy of ours may still be landing in shared memory when the CTA leaves
      if (!ok) {
        constexpr int N = BITS == 16 ? C::NST : C::NRAW;
        int at = BITS == 16 ? ring.i : raw.i;
        uint32_t ph = BITS == 16 ? ring.ph : raw.ph;
        for (int k = 0; k < min(issued, N); ++k) {
          if (--at < 0) {
            at += N;
            ph ^= 1u;
          }
          mbar_wait(BITS == 16 ? &b.full[at] : &b.rfull[at], ph, CH_WAIT);
        }
        if constexpr (BITS < 16) {
          for (int k = 0; k < min(scaled, C::NSC); ++k) {
            if (--keyed.i < 0) {
              keyed.i += C::NSC;
              keyed.ph ^= 1u;
            }
            mbar_wait(&b.scales[keyed.i], keyed.ph, CH_WAIT);
          }
        }
      }
    } else {
      // -------------------------------------------------------------- queries of a half (warps 10, 11)
      // 16 bytes a lane along the rows; rows past the last are zeros.  A half that sees no key of the piece takes
      // no part in its products and has none brought.
      const int w = warp - 10;
      uint8_t* qs = smem + C::QOFF + w * C::TILE;
      constexpr int LPR = D / 8, RPI = 32 / LPR;  // lanes of a row, rows of a warp's copy
      const int c = lane % LPR;
      uint32_t ph = 1u;
      // from a row to the one RPI rows on: steps of tokens and heads, a wrap of the heads at most (with a division and
      // products per row the first scores of a tile came 8100 cycles after the last ones' results, instead of 4600)
      const int dt = RPI / a.group, dg = RPI - dt * a.group;
      const int64_t step = dt * a.q_ts + dg * a.q_hs, wrap = a.q_ts - a.group * a.q_hs;
      JobReader reader(jobs, b);
      Job job;
      while (ok) {
        ok = reader.next(job);
        if (job.tiles < 0) break;
        const int rows = job.n * a.group - job.tile * CH_ROWS - w * 128;
        if (rows <= 0 || (w ? job.tiles : job.tiles0) == 0) continue;
        if (!mbar_wait(&b.qfree[w], ph, CH_WAIT)) {
          ok = false;
          break;
        }
        ph ^= 1u;
        const uint32_t row0 = job.tile * CH_ROWS + w * 128 + lane / LPR;
        const uint32_t i = row0 / static_cast<uint32_t>(a.group);  // token and head of the row
        int g = row0 - i * a.group;
        const T* base = static_cast<const T*>(a.q) + job.start * a.q_ts + job.head * a.group * a.q_hs + c * 8;
        const T* src = base + i * a.q_ts + g * a.q_hs;
#pragma unroll 8
        for (int r = lane / LPR; r < 128; r += RPI) {
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(qs + chunk_off(r, c))),
                       "l"(r < rows ? src : base), "r"(r < rows ? 16 : 0)
                       : "memory");
          src += step;
          g += dg;
          if (g >= a.group) {
            g -= a.group;
            src += wrap;
          }
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
        fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&b.qfull[w]);
      }
    }
  } else {
    // ---------------------------------------------------------------- codes -> 16-bit operand tiles
    if constexpr (BITS < 16) {
      regs_fewer<64>();
      constexpr int PPR = D / 16;  // 16-code pieces of a row
      // four warps turn keys, four values: while one group waits for its stores to be visible to the tensor
      // core, the other works
      const int tid = (threadIdx.x - 384) & 127, kv = (warp - 12) >> 2;
      const int col = tid % PPR, r0 = tid / PPR;
      int at = kv;  // place in the ring of operand tiles: keys even, values odd
      uint32_t ph = 0, rph = 0;
      JobReader reader(jobs, b);
      Job job;
      while (ok) {
        ok = reader.next(job);
        if (job.tiles < 0) break;
        for (int j = 0; j < job.tiles; ++j) {
          const int rest = job.kend - job.key0 - j * CH_KEYS;
          if (!mbar_wait(&b.empty[at], ph ^ 1u, CH_WAIT)) {
            ok = false;
            break;
          }
          uint8_t* tile = smem + C::RING + at * C::TILE;
          if (kv && !mbar_wait(&b.scales[at >> 1], ph, CH_WAIT)) {
            ok = false;
            break;
          }
          float* scales = reinterpret_cast<float*>(smem + C::SCALES) + ((at >> 1) * 2 + 1) * CH_KEYS;  // of the values
          // A thread's pieces: NA of each half, STEP rows apart, N at a time (all at once, their instructions twice in the
          // cache: prompts of 2048 over 8 bits 357 us, 346 so).
          constexpr int STEP = 128 / PPR, NA = CH_RAW / STEP, N = NA / 2;
          constexpr int WORDS = BITS / 2;  // of a piece
          for (int hf = 0; hf < 2; ++hf) {
            const int rs = 2 * kv + hf;
            if (!mbar_wait(&b.rfull[rs], rph, CH_WAIT)) {
              ok = false;
              break;
            }
            const uint8_t* src = smem + C::ROFF + rs * C::RAW;
            uint8_t* dst = tile + hf * CH_RAW * 128;
            const int left = rest - hf * CH_RAW;
#pragma unroll 1
            for (int r1 = r0; r1 < CH_RAW; r1 += N * STEP) {
              uint32_t wd[N][WORDS];
              float sc[N], zf[N];
#pragma unroll
              for (int x = 0; x < N; ++x) {
                const int r = r1 + x * STEP;
                if constexpr (BITS == 8)
                  *reinterpret_cast<uint4*>(wd[x]) = *reinterpret_cast<const uint4*>(src + r * C::ROW + col * 16);
                else
                  *reinterpret_cast<uint2*>(wd[x]) = *reinterpret_cast<const uint2*>(src + r * C::ROW + col * 8);
                // values past the last: zeros (keys there: scores that no row sees)
                sc[x] = KEY_STEP;
                if (kv) sc[x] = r < left ? power_of(scales[hf * CH_RAW + r]) : 0.f;
                zf[x] = __uint_as_float(0x4B000000u | src[CH_RAW * C::ROW + r]);  // 2^23 + zero
              }
#pragma unroll
              for (int x = 0; x < N; ++x) {
                // (2^23 + code) s - (2^23 + zero) s: no step of it rounds, s being a power of two
                const float2 s2 = make_float2(sc[x], sc[x]), z2 = make_float2(-zf[x] * sc[x], -zf[x] * sc[x]);
                uint32_t out[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                  float2 f;
                  if constexpr (BITS == 8) {
                    const uint32_t v = wd[x][e >> 1];
                    f.x = __uint_as_float(__byte_perm(v, 0x4B000000u, 0x7650u + (e & 1) * 2));
                    f.y = __uint_as_float(__byte_perm(v, 0x4B000000u, 0x7651u + (e & 1) * 2));
                  } else {
                    const uint32_t v = wd[x][e >> 2] >> ((e & 3) * 8);
                    f.x = __uint_as_float((v & 15u) | 0x4B000000u);
                    f.y = __uint_as_float(((v >> 4) & 15u) | 0x4B000000u);
                  }
                  f = fma2(f, s2, z2);
                  if constexpr (FMT)  // bfloat16 holds it in the upper half
                    out[e] = __byte_perm(__float_as_uint(f.x), __float_as_uint(f.y), 0x7632u);
                  else
                    out[e] = pack2<T>(f.x, f.y);
                }
                // the columns of the second 64 elements store their odd chunk first: no two of 8 neighbours on a bank
                const int r = r1 + x * STEP;
                const bool o = (col & 4) != 0;
                const uint4 lo = make_uint4(out[0], out[1], out[2], out[3]), hi = make_uint4(out[4], out[5], out[6], out[7]);
                *reinterpret_cast<uint4*>(dst + chunk_off(r, 2 * col + (o ? 1 : 0))) = o ? hi : lo;
                *reinterpret_cast<uint4*>(dst + chunk_off(r, 2 * col + (o ? 0 : 1))) = o ? lo : hi;
              }
            }
            if (kv) {  // the parts of the scales, for the softmax: a row per lane, of those that the warp has converted
              constexpr int NB = 32 / PPR;
              __syncwarp();
              if (lane < NB * NA) {
                float* scale = scales + hf * CH_RAW + (tid >> 5) * NB + lane % NB + lane / NB * STEP;
                *scale = part_of(*scale);
              }
              __syncwarp();
              if (hf == 1 && lane == 0) mbar_arrive(&b.parts[at >> 1]);
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&b.rempty[rs]);
          }
          if (!ok) break;
          fence_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&b.full[at]);
          rph ^= 1u;
          if ((at += 2) >= C::NST) {
            at = kv;
            ph ^= 1u;
          }
        }
      }
    }
  }
  if (!ok) atomicExch(&g_chunk_status, kStatusTimeout);
  tc_fence_before();
  __syncthreads();
  if (threadIdx.x == 0) odd[blockIdx.x] = *any_odd;
  if (warp == 8) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
  wait_for_last();
}

// Where a CTA met an accumulator that is not finite, rows are looked at again: a value that a row does not
// see, NaN or infinite, has met its zero weight in the products.  One warp per (row, head) whose result
// is not finite works it out key by key over the keys it sees.  Otherwise the launch reads the CTAs'
// words and ends.
template <typename T, int D, int BITS>
__global__ void __launch_bounds__(128) chunk_redo_kernel(const Args a, const int* __restrict__ odd, int n) {
  const int lane = threadIdx.x & 31;
  int any = 0;
  next_may_start();
  wait_for_last();
  for (int x = threadIdx.x; x < n; x += 128) any |= odd[x];
  if (!__syncthreads_or(any)) return;
  const int64_t all = static_cast<int64_t>(a.tokens) * a.heads;
  for (int64_t w = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 5); w < all; w += gridDim.x * 4) {
    const int t = static_cast<int>(w / a.heads), h = static_cast<int>(w % a.heads);
    int lo = 0, hi = a.seqs;  // the last sequence that starts at or before t
    while (hi - lo > 1) {
      const int mid = (lo + hi) / 2;
      (__ldg(a.starts + mid) <= t ? lo : hi) = mid;
    }
    const Seq q = sequence(a, lo);
    const int i = t - q.start;
    if (i < 0 || i >= q.n || static_cast<int64_t>(q.n) * a.group <= kStepRows) continue;
    T* o = static_cast<T*>(a.out) + w * D;
    bool fine = true;
#pragma unroll
    for (int c = 0; c < D / 32; ++c) fine = fine && fabsf(to_f32(o[lane + 32 * c])) < INFINITY;
    if (__all_sync(0xffffffffu, fine)) continue;
    float m, l, acc[D / 32];
    row_attention<T, D, BITS>(a, lo, h / a.group, static_cast<const T*>(a.q) + t * a.q_ts + h * a.q_hs, 0, seen(a, q, i), m,
                              l, acc);
    const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
    for (int c = 0; c < D / 32; ++c) o[lane + 32 * c] = to16<T>(acc[c] * inv);
  }
}

// ------------------------------------------------------------------ host
typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
  static EncodeTiledFn fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiledFn>(p);
  });
  return fn;
}

// The vectors of a 16-bit cache as rows; a box is 64 elements of the keys of a page (at most 128).
template <typename T>
int cache_map(CUtensorMap* m, const void* base, const Args& a, int d) {
  EncodeTiledFn enc = encode_fn();
  if (!enc) return GPTQ_ERR_CUDA;
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(d),
                              (static_cast<cuuint64_t>(a.pages) * a.kv_heads) << a.page_shift};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(d) * 2};
  const cuuint32_t box[2] = {64, static_cast<cuuint32_t>(std::min(1 << a.page_shift, CH_KEYS))};
  const cuuint32_t es[2] = {1, 1};
  const CUresult r = enc(m, std::is_same<T, __half>::value ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
                         2, const_cast<void*>(base), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
                         CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? GPTQ_OK : GPTQ_ERR_CUDA;
}

template <typename T, int D, int BITS>
int run(const Args& a, int grid, float* part, Cut* cut, int* odd, bool next, cudaStream_t s) {
  using C = Cfg<D, BITS>;
  GPTQ_TRY(ensure_smem_limit(reinterpret_cast<const void*>(chunk_kernel<T, D, BITS>), C::SMEM));
  CUtensorMap tk = {}, tv = {};
  if (BITS == 16) {
    GPTQ_TRY(cache_map<T>(&tk, a.kc, a, D));
    GPTQ_TRY(cache_map<T>(&tv, a.vc, a, D));
  }
  if (next) return launch_next(chunk_kernel<T, D, BITS>, dim3(grid), C::THREADS, C::SMEM, s, tk, tv, a, part, cut, odd);
  chunk_kernel<T, D, BITS><<<grid, C::THREADS, C::SMEM, s>>>(tk, tv, a, part, cut, odd);
  return after_launch();
}

template <typename T, int D>
int redo(const Args& a, int bits, const int* odd, int n, cudaStream_t s) {
  if (bits == 16) return launch_next(chunk_redo_kernel<T, D, 16>, dim3(n), 128, 0, s, a, odd, n);
  if (bits == 8) return launch_next(chunk_redo_kernel<T, D, 8>, dim3(n), 128, 0, s, a, odd, n);
  return launch_next(chunk_redo_kernel<T, D, 4>, dim3(n), 128, 0, s, a, odd, n);
}

}  // namespace

int run_chunk(const Args& a, int dtype, int head_dim, int bits, int grid, float* part, Cut* cut, int* odd, bool next,
              cudaStream_t s) {
#define GPTQ_CHUNK(T, D)                                                                                       \
  return bits == 16  ? run<T, D, 16>(a, grid, part, cut, odd, next, s)                                          \
         : bits == 8 ? run<T, D, 8>(a, grid, part, cut, odd, next, s)                                           \
                     : run<T, D, 4>(a, grid, part, cut, odd, next, s)
  if (dtype == GPTQ_BF16) {
    if (head_dim == 128) GPTQ_CHUNK(__nv_bfloat16, 128);
    GPTQ_CHUNK(__nv_bfloat16, 64);
  }
  if (head_dim == 128) GPTQ_CHUNK(__half, 128);
  GPTQ_CHUNK(__half, 64);
#undef GPTQ_CHUNK
}

int run_chunk_redo(const Args& a, int dtype, int head_dim, int bits, const int* odd, int n, cudaStream_t s) {
  if (dtype == GPTQ_BF16)
    return head_dim == 128 ? redo<__nv_bfloat16, 128>(a, bits, odd, n, s) : redo<__nv_bfloat16, 64>(a, bits, odd, n, s);
  return head_dim == 128 ? redo<__half, 128>(a, bits, odd, n, s) : redo<__half, 64>(a, bits, odd, n, s);
}

int chunk_device_status(int clear) {
  int h = 0;
  if (cudaMemcpyFromSymbol(&h, g_chunk_status, sizeof(int)) != cudaSuccess) return GPTQ_ERR_CUDA;
  if (clear && h != GPTQ_OK) {
    const int z = 0;
    cudaMemcpyToSymbol(g_chunk_status, &z, sizeof(int));
  }
  return h;
}

}  // namespace paged
}  // namespace gptq
