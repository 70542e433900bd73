// How the keys of a batch are shared among CTAs.  The sequences that a kernel takes (by their number
// of rows) stand in a line, each as kv_heads x units of keys; the line is cut into equal shares, one
// per CTA.  The lengths live on the device, so every CTA works the cut out for itself.
#pragma once

#include "paged.cuh"

namespace gptq {
namespace paged {

struct Share {
  int grid;
  int whole;             // not 0: no cutting, teams of so many CTAs (a cluster) take whole items
  int min_per;           // least units of a share
  int rows_lo, rows_hi;  // the sequences taken: rows (tokens x heads of a kv head) in this range
};

struct Cursor {
  int64_t at, end;  // position on the line (units; items where whole), and where the share ends
  int64_t per;      // units of a share
  int s, head, u0, u1, units;
};

__device__ __forceinline__ int units_of(const Args& a, const Share& sh, int unit, int s) {
  const Seq q = sequence(a, s);
  const int64_t rows = static_cast<int64_t>(q.n) * a.group;
  if (rows < sh.rows_lo || rows > sh.rows_hi) return 0;
  return max(1, (q.len + unit - 1) / unit);  // no keys: a piece that writes zeros
}

__device__ __forceinline__ int64_t shfl_up64(int64_t v, int o) { return __shfl_up_sync(0xffffffffu, v, o); }

// Inclusive sum over the block; every thread also gets the total.  ws: THREADS / 32 words of shared memory.
template <int THREADS>
__device__ __forceinline__ int64_t block_scan(int64_t v, int64_t& total, int64_t* ws) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t x = shfl_up64(v, o);
    if (lane >= o) v += x;
  }
  __syncthreads();
  if (lane == 31) ws[warp] = v;
  __syncthreads();
  total = 0;
#pragma unroll
  for (int w = 0; w < THREADS / 32; ++w) {
    if (w < warp) v += ws[w];
    total += ws[w];
  }
  return v;
}

__device__ __forceinline__ int64_t share_of(const Share& sh, int64_t line) {
  return max((line + sh.grid - 1) / sh.grid, static_cast<int64_t>(sh.min_per));
}

__device__ __forceinline__ void set_whole(const Args& a, const Share& sh, int unit, Cursor& c) {
  const int rank = blockIdx.x % sh.whole;
  for (; c.at < c.end; c.at += sh.grid / sh.whole) {
    c.s = static_cast<int>(c.at / a.kv_heads);
    c.head = static_cast<int>(c.at - static_cast<int64_t>(c.s) * a.kv_heads);
    c.units = units_of(a, sh, unit, c.s);
    c.u0 = static_cast<int>(static_cast<int64_t>(c.units) * rank / sh.whole);
    c.u1 = static_cast<int>(static_cast<int64_t>(c.units) * (rank + 1) / sh.whole);
    if (c.units) return;
  }
}

// The first piece of this CTA's share; false if it has none.  All threads.
template <int THREADS>
__device__ bool first_piece(const Args& a, const Share& sh, int unit, Cursor& c, Cursor* shared) {
  __shared__ int64_t ws[THREADS / 32];
  if (sh.whole) {
    c.at = blockIdx.x / sh.whole;
    c.end = static_cast<int64_t>(a.seqs) * a.kv_heads;
    set_whole(a, sh, unit, c);
    return c.at < c.end;
  }
  int64_t all = 0, total;
  for (int x = threadIdx.x; x < a.seqs; x += THREADS) all += units_of(a, sh, unit, x);
  const int64_t upto = block_scan<THREADS>(all, total, ws) * a.kv_heads;
  total *= a.kv_heads;
  const int64_t per = share_of(sh, total);
  c.per = per;
  c.at = blockIdx.x * per;
  c.end = min(total, c.at + per);
  if (c.at >= c.end) return false;
  auto take = [&](int x, int64_t u, int64_t lo) {
    if (u && lo <= c.at && c.at < lo + u) {
      const int64_t per_head = u / a.kv_heads, rem = c.at - lo;
      shared->s = x;
      shared->units = static_cast<int>(per_head);
      shared->head = static_cast<int>(rem / per_head);
      shared->u0 = static_cast<int>(rem % per_head);
    }
  };
  if (a.seqs <= THREADS) {
    take(threadIdx.x, all * a.kv_heads, upto - all * a.kv_heads);
  } else {
    int64_t base = 0;
    for (int x0 = 0; x0 < a.seqs; x0 += THREADS) {
      const int x = x0 + threadIdx.x;
      const int64_t u = x < a.seqs ? static_cast<int64_t>(units_of(a, sh, unit, x)) * a.kv_heads : 0;
      int64_t sum;
      const int64_t incl = block_scan<THREADS>(u, sum, ws);
      take(x, u, base + incl - u);
      base += sum;
      if (base > c.at) break;
    }
  }
  __syncthreads();
  c.s = shared->s;
  c.units = shared->units;
  c.head = shared->head;
  c.u0 = shared->u0;
  c.u1 = static_cast<int>(min(static_cast<int64_t>(c.units), c.u0 + (c.end - c.at)));
  return true;
}

__device__ __forceinline__ void next_piece(const Args& a, const Share& sh, int unit, Cursor& c) {
  if (sh.whole) {
    c.at += sh.grid / sh.whole;
    set_whole(a, sh, unit, c);
    return;
  }
  c.at += c.u1 - c.u0;
  if (c.at >= c.end) return;
  if (++c.head == a.kv_heads) {
    c.head = 0;
    do {
      ++c.s;
      c.units = units_of(a, sh, unit, c.s);
    } while (c.units == 0);
  }
  c.u0 = 0;
  c.u1 = static_cast<int>(min(static_cast<int64_t>(c.units), c.end - c.at));
}

}  // namespace paged
}  // namespace gptq
