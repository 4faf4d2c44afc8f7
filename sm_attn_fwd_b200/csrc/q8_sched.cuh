// How the 8-bit decode kernels share a batch of ragged sequences among their CTAs.
//
// A unit is one (sequence, KV head, tile of query rows); it has as many key tiles
// (128 keys) as its sequence.  All units' tiles, in the order (sequence, head, row
// tile), form one line of T tiles, and CTA c of G takes tiles [c T / G, (c + 1) T / G)
// (G = the number of CTAs, at most T; the rest get none): equal work whatever the
// lengths, one start-up per CTA, and a unit is cut only where a CTA's share ends, its
// pieces in neighbouring CTAs.  The lengths are known on the device only, so every
// CTA (and the combine) works its part out from kv_lens.
//
// A unit that one CTA computes whole is written to the outputs by it.  A CTA has at
// most two other pieces, the end of a unit that an earlier CTA began and the start
// of one that a later CTA ends: partial results in slots 2 c and 2 c + 1 of the
// workspace, merged by the combine kernel.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "attn_params.h"

namespace attn {
namespace q8 {

// A sequence's length in [0, Lk], and its key tiles.
__device__ __forceinline__ int seq_len(const int32_t* kv_lens, int b, int Lk) {
  return min(max(__ldg(kv_lens + b), 0), Lk);
}
__device__ __forceinline__ int tiles_of(int len) { return (int)(((long long)len + 127) >> 7); }

// Tiles of one unit per sequence summed over the batch (the whole warp calls it);
// sets *bad where an entry is out of range.
__device__ __forceinline__ long long sum_tiles(const int32_t* kv_lens, int B, int Lk, bool* bad) {
  const int lane = threadIdx.x & 31;
  long long n = 0;
  for (int b = lane; b < B; b += 32) {
    const int len = __ldg(kv_lens + b);
    if (len < 0 || len > Lk) *bad = true;
    n += tiles_of(min(max(len, 0), Lk));
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) n += __shfl_xor_sync(0xffffffffu, n, o);
  return n;
}

// The sequence whose units hold tile g of the line (units per sequence: `units`), and
// the line's tiles before that sequence (the whole warp calls it; g < T).
__device__ __forceinline__ int find_seq(const int32_t* kv_lens, int B, int Lk, int units,
                                        long long g, long long* before) {
  const int lane = threadIdx.x & 31;
  long long base = 0;
  for (int b0 = 0; b0 < B; b0 += 32) {
    const long long mine =
        b0 + lane < B ? (long long)tiles_of(seq_len(kv_lens, b0 + lane, Lk)) * units : 0;
    long long upto = mine;  // inclusive sum over the lanes
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long t = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += t;
    }
    const uint32_t past = __ballot_sync(0xffffffffu, base + upto > g);
    if (past != 0u) {
      const int l = __ffs(past) - 1;
      *before = base + __shfl_sync(0xffffffffu, upto - mine, l);
      return b0 + l;
    }
    base += __shfl_sync(0xffffffffu, upto, 31);
  }
  *before = base;
  return B;  // not reached for g < T
}

// CTAs that take part for T > 0 tiles; the first tile of CTA c, and the CTA that holds
// tile g, over G <= T CTAs.
__device__ __forceinline__ int ctas_used(long long T, int ctas) {
  return T < ctas ? (int)T : ctas;
}
__device__ __forceinline__ long long first_tile(long long c, long long T, int G) {
  return c * T / G;
}
__device__ __forceinline__ long long cta_of(long long g, long long T, int G) {
  return ((g + 1) * G - 1) / T;
}

// A CTA's share: tiles [g0, g1) of the line, starting in unit (b, h) of base `base`.
struct Share {
  long long g0, g1, base;
  int b, h;
};

// Worked out by one whole warp.
__device__ __forceinline__ Share find_share(const int32_t* kv_lens, int B, int Lk, int units,
                                            int cta, int ctas, int* err) {
  bool bad = false;
  const long long T = sum_tiles(kv_lens, B, Lk, &bad) * units;
  if (bad && cta == 0) atomicOr(err, kDevErrBadKvLen);
  Share s;
  s.g0 = s.g1 = s.base = 0;
  s.b = s.h = 0;
  const int G = ctas_used(T, ctas);
  if (cta < G) {
    s.g0 = first_tile(cta, T, G);
    s.g1 = first_tile(cta + 1, T, G);
    s.b = find_seq(kv_lens, B, Lk, units, s.g0, &s.base);
    const int tiles = tiles_of(seq_len(kv_lens, s.b, Lk));
    s.h = (int)((s.g0 - s.base) / tiles);
    s.base += (long long)s.h * tiles;
  }
  return s;
}

// Walks the pieces of a share: tiles [t0, t1) of `tiles` of unit (b, h).
struct Walk {
  long long g1, base;
  int b, h, len, tiles, t0, t1;

  __device__ __forceinline__ void start(const Share& s, const int32_t* kv_lens, int Lk) {
    g1 = s.g1;
    base = s.base;
    b = s.b;
    h = s.h;
    t0 = t1 = 0;
    tiles = len = 0;
    if (s.g0 >= s.g1) return;
    len = seq_len(kv_lens, b, Lk);
    tiles = tiles_of(len);
    t0 = (int)(s.g0 - base);
    t1 = (int)min((long long)tiles, g1 - base);
  }
  __device__ __forceinline__ bool valid() const { return t0 < t1; }
  // the next piece; valid() is false after the last
  __device__ __forceinline__ void next(const int32_t* kv_lens, int Lk, int units) {
    base += tiles;
    t0 = t1 = 0;
    if (base >= g1) return;
    if (++h == units) {
      h = 0;
      do {  // a later sequence has tiles: base < g1 <= T
        len = seq_len(kv_lens, ++b, Lk);
      } while (len == 0);
      tiles = tiles_of(len);
    }
    t1 = (int)min((long long)tiles, g1 - base);
  }
  __device__ __forceinline__ bool whole() const { return t0 == 0 && t1 == tiles; }
  __device__ __forceinline__ int slot(int cta) const { return 2 * cta + (t0 > 0 ? 0 : 1); }
};

}  // namespace q8
}  // namespace attn
