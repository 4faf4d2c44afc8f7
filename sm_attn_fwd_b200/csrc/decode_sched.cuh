// How the 8-bit decode kernels share a batch of ragged sequences among their CTAs.
//
// A unit is one (sequence, KV head, tile of query rows); it has as many key tiles
// (128 keys) as its sequence.  A unit with n > 0 tiles costs n + piece: starting on and
// finishing a unit takes about as long as `piece` tiles (piece_tiles() in
// decode_params.h; with 28 one-tile units in one CTA and 28 tiles of two units in
// another, a batch of ragged lengths from 1 to 4099 took 49 us where one of equal lengths
// and more tiles took 30).  All units, in
// the order (sequence, head, row tile), form one line of length T, and CTA c of G
// takes [c T / G, (c + 1) T / G) of it (G = the number of CTAs, at most T; the rest get
// nothing): equal work whatever the lengths, one start-up per CTA, and a unit is cut
// only where a CTA's share ends, its pieces in neighbouring CTAs.  Tile t of a unit
// that starts at `base` lies at base + piece + t.  The lengths are known on the device
// only, so every CTA (and the combine) works its part out from kv_lens.
//
// A unit that one CTA computes whole is written to the outputs by it.  A CTA has at
// most two other pieces, the end of a unit that an earlier CTA began and the start
// of one that a later CTA ends: partial results in slots 2 c and 2 c + 1 of the
// workspace, merged by the combine kernel.
//
// T < 2^31 is checked on the host.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "attn_params.h"
#include "decode_params.h"

namespace attn {
namespace sched {

// A sequence's length in [0, Lk], its key tiles, and the cost of a unit of it.
__device__ __forceinline__ int seq_len(const int32_t* kv_lens, int b, int Lk) {
  return min(max(__ldg(kv_lens + b), 0), Lk);
}
__device__ __forceinline__ int tiles_of(int len) { return (int)(((unsigned)len + 127u) >> 7); }
__device__ __forceinline__ int cost_of(int len, int piece) {
  return len > 0 ? tiles_of(len) + piece : 0;
}

// [first(c), first(c + 1)) is CTA c's part of a line of length T over G <= T CTAs, the
// first T % G of them one longer; of(x) is the CTA that holds x.
struct Split {
  int q, r;
  __device__ __forceinline__ Split(int T, int G) : q(T / G), r(T - T / G * G) {}
  __device__ __forceinline__ int first(int c) const { return c * q + min(c, r); }
  __device__ __forceinline__ int of(int x) const {
    const int longer = r * (q + 1);
    return x < longer ? x / (q + 1) : r + (x - longer) / q;
  }
};
__device__ __forceinline__ int ctas_used(int T, int ctas) { return min(T, ctas); }

// A CTA's share [g0, g1) of the line, starting in unit (b, h), which starts at `base`.
struct Share {
  int g0, g1, base;
  int b, h, piece;
};

// Walks the pieces of a share: tiles [t0, t1) of the `tiles` of unit (b, h).
struct Walk {
  int g1, base, piece;
  int b, h, len, tiles, t0, t1;

  __device__ __forceinline__ void start(const Share& s, const int32_t* kv_lens, int Lk) {
    g1 = s.g1;
    piece = s.piece;
    base = s.base;
    b = s.b;
    h = s.h;
    t0 = t1 = 0;
    tiles = len = 0;
    if (s.g0 >= s.g1) return;
    len = seq_len(kv_lens, b, Lk);
    tiles = tiles_of(len);
    t0 = max(0, s.g0 - base - piece);
    t1 = min(tiles, max(0, g1 - base - piece));
  }
  // false after the last piece (and for a share that ends before a unit's first tile)
  __device__ __forceinline__ bool valid() const { return t0 < t1; }
  __device__ __forceinline__ void next(const int32_t* kv_lens, int Lk, int units) {
    base += tiles + piece;
    t0 = t1 = 0;
    if (base >= g1) return;
    if (++h == units) {
      h = 0;
      do {  // a later sequence has tiles: base < g1 <= T
        len = seq_len(kv_lens, ++b, Lk);
      } while (len == 0);
      tiles = tiles_of(len);
    }
    t1 = min(tiles, max(0, g1 - base - piece));
  }
  __device__ __forceinline__ bool whole() const { return t0 == 0 && t1 == tiles; }
  __device__ __forceinline__ int slot(int cta) const { return 2 * cta + (t0 > 0 ? 0 : 1); }
};

// The share of CTA `cta`, worked out by one whole warp; flags lengths out of range.
__device__ __forceinline__ Share find_share(const int32_t* kv_lens, int B, int Lk, int units,
                                            int piece, int cta, int ctas, int* err) {
  const int lane = threadIdx.x & 31;
  bool bad = false;
  int sum = 0;
#pragma unroll 4  // the loads of four rounds in flight together
  for (int b = lane; b < B; b += 32) {
    const int len = __ldg(kv_lens + b);
    if (len < 0 || len > Lk) bad = true;
    sum += cost_of(min(max(len, 0), Lk), piece);
  }
  if (bad && cta == 0) atomicOr(err, kDevErrBadKvLen);
  const int T = __reduce_add_sync(0xffffffffu, sum) * units;
  Share s = {0, 0, 0, 0, 0, piece};
  const int G = ctas_used(T, ctas);
  if (cta >= G) return s;
  const Split split(T, G);
  s.g0 = split.first(cta);
  s.g1 = split.first(cta + 1);
  // the sequence that holds g0
  for (int b0 = 0; b0 < B; b0 += 32) {
    const int mine = b0 + lane < B ? cost_of(seq_len(kv_lens, b0 + lane, Lk), piece) * units : 0;
    int upto = mine;  // inclusive sum over the lanes
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int t = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += t;
    }
    const uint32_t past = __ballot_sync(0xffffffffu, s.base + upto > s.g0);
    if (past != 0u) {
      const int l = __ffs(past) - 1;
      s.b = b0 + l;
      s.base += __shfl_sync(0xffffffffu, upto - mine, l);
      const int cost = __shfl_sync(0xffffffffu, mine, l) / units;
      s.h = (s.g0 - s.base) / cost;
      s.base += s.h * cost;
      break;
    }
    s.base += __shfl_sync(0xffffffffu, upto, 31);
  }
  return s;
}

// The key tiles of a share.
__device__ __forceinline__ int count_tiles(const Share& s, const int32_t* kv_lens, int Lk,
                                           int units) {
  int n = 0;
  Walk w;
  for (w.start(s, kv_lens, Lk); w.valid(); w.next(kv_lens, Lk, units)) n += w.t1 - w.t0;
  return n;
}

// Lets the kernel that follows in the stream start launching (it waits for this one's
// results itself).
__device__ __forceinline__ void let_next_kernel_launch() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

}  // namespace sched
}  // namespace attn
