// Decode over an 8-bit cache for many query rows per KV head (group * Lq up to 128
// per tile), for sm_100a: the tensor-memory counterpart of attn_decode_rows.cu.
//
// With 8 query rows a key's codes are used 8 times and the register path of
// attn_decode_rows.cu keeps up with memory; with 128 rows (16 drafted tokens x 8
// heads) the products are 16 times larger and belong on tcgen05.  Its operands
// must lie in shared or tensor memory as 16-bit values, so here the codes are
// expanded: four warpgroups turn the K and V tiles, as TMA left them, into the bf16
// tiles the bf16 decode would have loaded.
//
//   K'_j = kc_j 2^(ke_j - kref),  V'_j = vc_j 2^(ve_j - vref),
// kref and vref the tile's largest scale bytes.  Both are exact in bf16 (4
// significant bits), so the only roundings are P's and O's.  kref joins the tile's
// softmax scale, c_t = scale log2 e 2^(kref - 127); vref joins the exponent of
// P' = 2^(s c_t - m + vref - 127), and the row sum gets sum(P') 2^(127 - vref).
// Neither costs the softmax an instruction per score.
//
// Expanding two codes: a byte permute sign-extends them into two 16-bit halves, a
// shift by 4 and a mask leave s 0000 eeee mmm 0000, which read as bf16 is the value
// times 2^-120 (e4m3 subnormals included), and one packed multiply by
// 2^(120 + e - ref) finishes them: 4 instructions per pair.  A factor of 0 clears
// keys past the end, whatever their codes hold.  The construction makes NaN codes
// finite, so the expansion also looks for them (a mask and an add per four codes) and
// notes the tile; the end of a piece with such a tile looks its codes up again and gives
// its rows (NaN in a key) or columns (NaN in a value) NaN.  That leaves the expansion
// without a branch: 16 x 8 KV heads, up to 32768 keys, 128 query rows take 297 us
// instead of 294, and 315 where it writes the NaN itself.
//
// Roles (896 threads, one CTA per SM, looping over the pieces of its share of the
// work, decode_sched.cuh): warp 0 loads the codes, in half tiles of 64 keys; warp 1
// issues the MMAs; warp 2 loads Q; warp 3 turns scale bytes into factors (loading them
// where they are used stalled the expansion 800 cycles per tile); warpgroups 1 and 2 are
// the softmaxes, one for the first 64 keys of every tile and one for the last, each with a
// running maximum and an O of its own in tensor memory, so that they exchange
// nothing; S is double buffered, the next tile's ready while this one is worked on;
// warpgroups 3 to 6 expand the halves of the K and the V tiles.  At the end of a piece
// warpgroup 1 merges the two O and writes the result, while the loads, the expansion
// and the first S of the next piece go on.
//
// What bounds it: per 128-key tile at d = 128 shared memory moves 32 KB of codes in,
// 32 KB out to the expansion, 64 KB back and 96 KB to the MMAs, 1750 cycles at 128
// bytes a cycle, against 1400 cycles that the codes take to arrive at the SM's share
// of the copy bandwidth and 1024 each for the MMAs and the exponentials.  It takes about
// 3000: a softmax's chain per tile (wait, load of S, maximum, exponentials, store of
// P) and the expansion's share of the issue slots; with the expansion's arithmetic left
// out it still takes 94 % of the time.  Measured: 16 x 8 KV heads x 16384 keys, 128 query
// rows: 208 us (2.6 TB/s); up to 32768 keys in 16-key pages: 296 us, where bytes and
// products each need 104.  One softmax per even and odd tile, whose S waits for the P V
// before it, with one expansion warpgroup for K and one for V: 313 us; this one with
// two expansion warpgroups: 306.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "attn_params.h"
#include "cache_q8.cuh"
#include "decode_params.h"
#include "host_once.h"
#include "ptx.cuh"
#include "decode_sched.cuh"
#include "softmax_row.cuh"

namespace attn {
namespace {

constexpr int kThreads = 896;
// registers per thread of the warpgroups: loads and MMAs; softmax (two); expansion (four).
// 48 + 2 * 120 + 4 * 48 <= 7 * 72, the launch's.
constexpr int kRegsIssue = 48;
constexpr int kRegsExpand = 48;
constexpr int kRegsSoftmax = 120;
// more than the launch's registers would wait for ever
static_assert(kRegsIssue + 2 * kRegsSoftmax + 4 * kRegsExpand <= 7 * 72, "register shares");
constexpr int kTmemCols = 512;
constexpr float kRescaleThreshold = 8.0f;  // log2 units
constexpr float kLn2 = 0.69314718055994530942f;
constexpr int kRefSlots = 8;     // tiles whose reference scales are kept
constexpr int kFactorSlots = 2;  // tiles of expansion factors

template <int D>
struct WCfg {
  static constexpr int kAtoms = D / 64;
  static constexpr int kAtomBytes = 128 * 128;
  static constexpr int kTileBytes = 128 * D * 2;   // an expanded tile (and Q)
  static constexpr int kRawBytes = 64 * D;         // a half tile of codes
  static constexpr int kStages = D == 64 ? 4 : 2;  // expanded K and V tiles each
  static constexpr int kRaw = D == 64 ? 8 : 4;     // half tiles of codes, K and V each
  static constexpr int kOffQ = 0;
  static constexpr int kOffK = kOffQ + kTileBytes;
  static constexpr int kOffV = kOffK + kStages * kTileBytes;
  static constexpr int kOffRaw = kOffV + kStages * kTileBytes;  // K's ring, then V's
  static constexpr int kOffMl = kOffRaw + 2 * kRaw * kRawBytes;  // (m, l) of the odd tiles
  // factors of the keys of a tile, as bf16 exponents: K's 128, then V's
  static constexpr int kOffFactor = kOffMl + 1024;
  static constexpr int kOffMisc = kOffFactor + kFactorSlots * 256;
  static constexpr int kOffBar = kOffMisc + 48 + kRefSlots * 8;
  static constexpr int kNumBars = 17 + 2 * kFactorSlots + 4 * kRaw + 4 * kStages;
  static constexpr int kSmemBytes = kOffBar + kNumBars * 8;
  static constexpr int kSmemAlloc = kSmemBytes + 1024;
  static_assert(kSmemAlloc <= 227 * 1024, "shared memory");
};

// 64 of a row's scores: P = 2^(s c - m) as packed bf16 pairs, returning their fp32 sum
// (row::exp2_pack128 on half a row).
__device__ __forceinline__ float exp2_pack64(const float (&s)[64], float c, float m,
                                             uint32_t (&pk)[32]) {
  constexpr int kAhead = 4;
  float e0[kAhead], e1[kAhead];
  float sum8[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) sum8[k] = 0.0f;
#pragma unroll
  for (int i = 0; i < 32 + kAhead; ++i) {
    if (i >= kAhead) {
      const int j = i - kAhead;
      const float p0 = e0[j % kAhead], p1 = e1[j % kAhead];
      ptx::add2_acc(sum8[(j & 3) * 2], sum8[(j & 3) * 2 + 1], p0, p1);
      pk[j] = ptx::pack_bf16x2(p0, p1);
    }
    if (i < 32) {
      float a0, a1;
      ptx::fma2_bc(a0, a1, s[2 * i], s[2 * i + 1], c, -m);
      e0[i % kAhead] = ptx::ex2(a0);
      e1[i % kAhead] = ptx::ex2(a1);
    }
  }
#pragma unroll
  for (int k = 0; k < 4; ++k) sum8[k] += sum8[k + 4];
  return (sum8[0] + sum8[1]) + (sum8[2] + sum8[3]);
}

// The largest of 64 scores, in 8 chains.
__device__ __forceinline__ float row_max64(const float (&v)[64]) {
  float m[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) m[j] = fmaxf(v[j], v[8 + j]);
#pragma unroll
  for (int i = 16; i < 64; i += 8)
#pragma unroll
    for (int j = 0; j < 8; ++j) m[j] = fmaxf(m[j], v[i + j]);
#pragma unroll
  for (int w = 4; w >= 1; w >>= 1)
#pragma unroll
    for (int j = 0; j < w; ++j) m[j] = fmaxf(m[j], m[j + w]);
  return m[0];
}

// O (+)= P V over 64 keys: 4 MMAs, P in tensor memory (8 columns per 16 keys), V
// MN-major in shared memory (2048 bytes per 16 keys).
__device__ __forceinline__ void mma_pv_chain4(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc,
                                              uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred e, p, one;\n\t.reg .b64 b;\n\t.reg .b32 a;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "setp.eq.u32 one, 0, 0;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t"
      "add.u32 a, %1, 8;   add.s64 b, %2, 128;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %3, one;\n\t"
      "add.u32 a, %1, 16;  add.s64 b, %2, 256;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %3, one;\n\t"
      "add.u32 a, %1, 24;  add.s64 b, %2, 384;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %3, one;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// Looks for NaN codes among keys [k0, k1) of sequence b and KV head hkv, by one whole warp.
// Bit 16: a key has one (the same in all lanes).  Bits 0 to 15 of lane l: the columns of
// chunk l % (D / 16), 16 of them, that a value has one in.
template <int D>
__device__ __noinline__ uint32_t find_nan(const DecodeParams& p, int b, int hkv, int k0, int k1) {
  constexpr int kChunks = D / 16;
  const int lane = threadIdx.x & 31;
  uint32_t cols = 0, keys = 0;
#pragma unroll 1
  for (int j = k0 + lane / kChunks; j < k1; j += 32 / kChunks) {
    long long row = ((long long)b * p.Hkv + hkv) * p.Lk + j;
    if (p.block_table) {
      const int page =
          __ldg(p.block_table + (long long)b * p.pages_per_seq + (j >> p.page_shift));
      if (page < 0 || page >= p.num_pages) continue;  // reads as zeros
      row = (((long long)page * p.Hkv + hkv) << p.page_shift) + (j & (p.page_size - 1));
    }
    const long long at = row * kChunks + lane % kChunks;
    const uint4 kw = reinterpret_cast<const uint4*>(p.k_codes)[at];
    const uint4 vw = reinterpret_cast<const uint4*>(p.v_codes)[at];
    const uint32_t k[4] = {kw.x, kw.y, kw.z, kw.w}, v[4] = {vw.x, vw.y, vw.z, vw.w};
#pragma unroll 1
    for (int i = 0; i < 16; ++i) {
      if ((k[i >> 2] >> (8 * (i & 3)) & 0x7fu) == 0x7fu) keys = 1u << 16;
      if ((v[i >> 2] >> (8 * (i & 3)) & 0x7fu) == 0x7fu) cols |= 1u << i;
    }
  }
  // lanes l, l + kChunks, ... have the same columns
#pragma unroll
  for (int x = kChunks; x < 32; x <<= 1) cols |= __shfl_xor_sync(0xffffffffu, cols, x);
  return cols | __reduce_or_sync(0xffffffffu, keys);
}

struct Misc {
  uint32_t tmem_base;
  int abort;
  uint32_t nan_end;  // 1 + the last tile that holds a NaN code of a live key, or 0
  int pad;
  sched::Share share;
  int total;
  float2 ref[kRefSlots];  // per tile: 2^(kref - 127), vref - 127
};
static_assert(sizeof(Misc) == 48 + kRefSlots * 8, "kOffBar");

enum : int {
  kQFull = 0,
  kQEmpty = 1,     // MMA -> Q loader: last S of the piece done
  kSFull = 2,      // [2] MMA -> both softmaxes: S of an even, odd tile
  // [x][j % 2], as a softmax can be two tiles ahead of the MMA issuer: a barrier's next
  // phase begins only after the wait for this one
  kPFull = 4,      // softmax x (128) -> MMA: its half of P written, its O rescaled
  kODone = 8,      // MMA -> softmax x: its P V of the tile done
  kOFree = 12,     // warpgroup 1 (128) -> MMA: both O read out
  kMlFull = 13,    // warpgroup 2 (128) -> warpgroup 1: its (m, l)
  kMlEmpty = 14,   // warpgroup 1 (128) -> warpgroup 2
  kDrain = 15,
  kPieceDone = 16, // MMA -> warpgroup 1: every P V of the piece done
  kFactorFull = 17,                           // [kFactorSlots] warp 3 -> expansion
  kFactorEmpty = kFactorFull + kFactorSlots,  // [kFactorSlots] expansion (8 warps) -> warp 3
  // raw_full[2][R], raw_empty[2][R] (K's, V's), then full[2][S], empty[2][S] of the expanded
  // tiles
  kRing = kFactorEmpty + kFactorSlots,
};

}  // namespace

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    attn_decode_q8_wide_kernel(const __grid_constant__ CUtensorMap tm_q,
                               const __grid_constant__ CUtensorMap tm_k,
                               const __grid_constant__ CUtensorMap tm_v,
                               const __grid_constant__ DecodeParams p) {
  using C = WCfg<D>;
  constexpr int S = C::kStages;
  constexpr int R = C::kRaw;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const uint32_t sq = ptx::smem_u32(smem + C::kOffQ);
  const uint32_t sk = ptx::smem_u32(smem + C::kOffK);
  const uint32_t sv_ = ptx::smem_u32(smem + C::kOffV);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::kOffBar);
  const uint32_t bar0 = ptx::smem_u32(bars);
  auto BAR = [bar0](int i) -> uint32_t { return bar0 + 8u * (uint32_t)i; };
  // kv: 0 = K, 1 = V
  auto RAW_FULL = [&](int kv, int i) { return BAR(kRing + kv * R + i); };
  auto RAW_EMPTY = [&](int kv, int i) { return BAR(kRing + 2 * R + kv * R + i); };
  auto FULL = [&](int kv, int st) { return BAR(kRing + 4 * R + kv * S + st); };
  auto EMPTY = [&](int kv, int st) { return BAR(kRing + 4 * R + 2 * S + kv * S + st); };
  Misc* misc = reinterpret_cast<Misc*>(smem + C::kOffMisc);
  volatile int* abort_flag = &misc->abort;
  int* err = p.err;
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int units = p.Hkv * p.row_tiles;
  const bool paged = p.block_table != nullptr;
  // pool index (page * Hkv + hkv) of the page that holds key j of (b, hkv), or -1
  auto pool = [&](int b, int hkv, int j) -> int {
    const int page =
        __ldg(p.block_table + (long long)b * p.pages_per_seq + (j >> p.page_shift));
    if (page < 0 || page >= p.num_pages) {
      atomicOr(err, kDevErrBadPage);
      return -1;
    }
    return page * p.Hkv + hkv;
  };

  if (warp == 0) {
    const sched::Share sh =
        sched::find_share(p.kv_lens, p.B, p.Lk, units, p.piece, blockIdx.x, gridDim.x, err);
    const int n = sched::count_tiles(sh, p.kv_lens, p.Lk, units);
    if (lane == 0) {
      misc->share = sh;
      misc->total = n;
      misc->abort = 0;
      misc->nan_end = 0;
    }
  } else if (warp == 1) {
    ptx::tmem_alloc(&misc->tmem_base, kTmemCols);
    ptx::tmem_relinquish();
  } else if (warp == 2) {
    if (lane == 0) {
      ptx::prefetch_tmap(&tm_q);
      ptx::prefetch_tmap(&tm_k);
      ptx::prefetch_tmap(&tm_v);
      ptx::mbar_init(&bars[kQFull], 1);
      ptx::mbar_init(&bars[kQEmpty], 1);
      for (int i = 0; i < 2; ++i) ptx::mbar_init(&bars[kSFull + i], 1);
      for (int i = 0; i < 4; ++i) {
        ptx::mbar_init(&bars[kPFull + i], 128);
        ptx::mbar_init(&bars[kODone + i], 1);
      }
      ptx::mbar_init(&bars[kOFree], 128);
      ptx::mbar_init(&bars[kMlFull], 128);
      ptx::mbar_init(&bars[kMlEmpty], 128);
      ptx::mbar_init(&bars[kDrain], 1);
      ptx::mbar_init(&bars[kPieceDone], 1);
      for (int i = 0; i < kFactorSlots; ++i) {
        ptx::mbar_init(&bars[kFactorFull + i], 1);
        ptx::mbar_init(&bars[kFactorEmpty + i], 16);
      }
      for (int i = 0; i < 2 * R; ++i) {
        ptx::mbar_init(&bars[kRing + i], 1);
        ptx::mbar_init(&bars[kRing + 2 * R + i], 4);
      }
      for (int i = 0; i < 2 * S; ++i) {
        ptx::mbar_init(&bars[kRing + 4 * R + i], 256);
        ptx::mbar_init(&bars[kRing + 4 * R + 2 * S + i], 1);
      }
      ptx::fence_mbar_init();
    }
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = misc->tmem_base;
  const sched::Share& share = misc->share;
  const int total = misc->total;  // key tiles of this CTA
  bool ok = true;

  if (warp < 4) {
    ptx::regs_dec<kRegsIssue>();
    if (warp == 0) {
      // ---------------------------------------------------------- TMA producer
      // One box per half tile of codes, or one per page slice (spread over the lanes)
      // for pages shorter than that; keys past the end read as zeros.
      const int rows = paged && p.page_size < 64 ? p.page_size : 64;
      const int n_box = 64 / rows;  // at most 4
      const uint64_t policy = ptx::l2_policy_evict_first();
      int hj = 0, n_k = 0;  // half tiles issued: V's hj, K's n_k
      sched::Walk w;
      for (w.start(share, p.kv_lens, p.Lk); w.valid() && ok; w.next(p.kv_lens, p.Lk, units)) {
        const int hkv = w.h / p.row_tiles;
        const int key_end = min(w.t1 * 128, w.len);
        auto half_pool = [&](int k0) -> int {
          if (!paged) return w.b * p.Hkv + hkv;
          const int key = k0 + lane * rows;
          return lane < n_box && key < key_end ? pool(w.b, hkv, key) : -1;
        };
        int z_next = half_pool(w.t0 * 128);
        for (int k0 = w.t0 * 128; k0 < w.t1 * 128; k0 += 64, ++hj) {
          const int slot = hj % R;
          const uint32_t ph = ((uint32_t)(hj / R) & 1u) ^ 1u;
          const int z = z_next;
          const int key = k0 + lane * rows;
          const int y = paged ? key & (p.page_size - 1) : key;
          for (int kv = 0; kv < 2; ++kv) {
            ok = ptx::mbar_wait_a(RAW_EMPTY(kv, slot), ph, abort_flag, err,
                                  kDevErrTimeoutProducer);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            uint64_t* bar = bars + kRing + kv * R + slot;
            if (lane == 0) ptx::mbar_arrive_expect_tx(bar, C::kRawBytes);
            __syncwarp();
            if (lane < n_box)
              ptx::tma_load_3d_hint(
                  smem + C::kOffRaw + (kv * R + slot) * C::kRawBytes + lane * rows * D,
                  kv ? &tm_v : &tm_k, bar, 0, y, z, policy);
            if (kv == 0) {
              n_k = hj + 1;
              if (k0 + 64 < w.t1 * 128) z_next = half_pool(k0 + 64);  // in flight meanwhile
            }
          }
          if (!ok) break;
        }
      }
      // Drain: every copy lands before the CTA exits (long done in a normal run).
      if (lane == 0) {
        for (int kv = 0; kv < 2; ++kv) {
          const int n = kv ? hj : n_k;
          for (int k = max(0, n - R); k < n; ++k) {
            int dummy = 0;
            ptx::mbar_wait_a(RAW_FULL(kv, k % R), (uint32_t)(k / R) & 1u, &dummy, nullptr, 0);
          }
        }
      }
    } else if (warp == 3) {
      // -------------------------------------------------------- scale factors
      // Lane l takes keys 4 l .. 4 l + 3 of a tile: one 32-bit word of scale bytes for K
      // and one for V, loaded kAhead tiles ahead of their use (page ids one more), as a
      // load from memory can take longer than a tile (3 ahead: no faster, 5 % slower in
      // one measurement).
      constexpr int kAhead = 2;
      sched::Walk a;  // of the tile whose page ids load next
      a.start(share, p.kv_lens, p.Lk);
      int at = a.t0;
      struct Tile {
        int key, n, z;  // the lane's first key, its live keys (0..4), and its pool index
      };
      auto fetch = [&]() -> Tile {  // the tile at `a`, which moves on
        Tile f = {0, 0, 0};
        if (!a.valid()) return f;
        const int hkv = a.h / p.row_tiles;
        f.key = at * 128 + 4 * lane;
        f.n = max(0, min(4, min(a.t1 * 128, a.len) - f.key));
        f.z = a.b * p.Hkv + hkv;
        if (paged && f.n > 0) f.z = pool(a.b, hkv, f.key);
        if (++at == a.t1) {
          a.next(p.kv_lens, p.Lk, units);
          at = a.t0;
        }
        return f;
      };
      // The scale bytes of a tile's keys, 0 past the end.  Words where they are aligned
      // and inside the row of the cache, else single bytes.
      auto load_word = [&](const uint8_t* exps, const Tile& f) -> uint32_t {
        if (f.n == 0 || f.z < 0) return 0u;
        const uint8_t* src =
            exps + (paged ? ((long long)f.z << p.page_shift) + (f.key & (p.page_size - 1))
                          : (long long)f.z * p.Lk + f.key);
        const bool inside = paged || f.key + 3 < p.Lk;
        if (inside && (reinterpret_cast<uintptr_t>(src) & 3) == 0)
          return __ldg(reinterpret_cast<const uint32_t*>(src));
        uint32_t w = 0;
        for (int i = 0; i < f.n; ++i) w |= (uint32_t)__ldg(src + i) << (8 * i);
        return w;
      };
      // Caps the four bytes of w and returns the largest one of the warp's; in 16-bit halves,
      // which have minimum and maximum instructions.
      auto cap_and_max = [](uint32_t& w) -> int {
        constexpr uint32_t kMax2 = (uint32_t)q8::kMaxScaleByte * 0x00010001u;
        const uint32_t even = __vminu2(w & 0x00ff00ffu, kMax2);
        const uint32_t odd = __vminu2(w >> 8 & 0x00ff00ffu, kMax2);
        w = even | odd << 8;
        const uint32_t m = __vmaxu2(even, odd);
        return (int)__reduce_max_sync(0xffffffffu, max(m & 0xffffu, m >> 16));
      };
      // bf16 exponents of 2^(120 + e - ref), 247 + e - ref, of four keys; 0 (a factor of
      // zero) past the end only.  One addition: no byte carries or becomes 0, as
      // e <= 247, e - 7 <= ref <= 246.
      auto factors = [](uint32_t w, uint32_t alive, int ref) -> uint32_t {
        return (w + (uint32_t)(247 - ref) * 0x01010101u) & alive;
      };
      uint32_t k[kAhead], v[kAhead], live[kAhead];  // live: mask of the live keys' bytes
      auto load = [&](const Tile& f, int i) {
        k[i] = load_word(p.k_exp, f);
        v[i] = load_word(p.v_exp, f);
        live[i] = f.n == 4 ? ~0u : (1u << (8 * f.n)) - 1u;
      };
#pragma unroll
      for (int i = 0; i < kAhead; ++i) load(fetch(), i);
      Tile f = fetch();
      for (int j = 0; j < total;) {
#pragma unroll
        for (int i = 0; i < kAhead; ++i, ++j) {
          if (j >= total) break;
          uint32_t kw = k[i] & live[i], vw = v[i] & live[i];
          const uint32_t alive = live[i];
          load(f, i);
          f = fetch();
          const int kref = min(max(cap_and_max(kw), 1), 246);
          // vref is bounded so that P' = p 2^(vref - 127) stays clear of both ends of fp32
          const int vref = min(max(cap_and_max(vw), 67), 240);
          const int fs = j % kFactorSlots;
          ok = ptx::mbar_wait_a(BAR(kFactorEmpty + fs), ((uint32_t)(j / kFactorSlots) & 1u) ^ 1u,
                                abort_flag, err, kDevErrTimeoutProducer);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          uint32_t* out = reinterpret_cast<uint32_t*>(smem + C::kOffFactor + fs * 256);
          out[lane] = factors(kw, alive, kref);
          out[32 + lane] = factors(vw, alive, vref);
          if (lane == 0)
            misc->ref[j % kRefSlots] =
                make_float2(__uint_as_float((uint32_t)kref << 23), (float)(vref - 127));
          __syncwarp();
          if (lane == 0) ptx::mbar_arrive_a(BAR(kFactorFull + fs));
        }
        if (!ok) break;
      }
    } else if (warp == 2) {
      // ---------------------------------------------------------- Q of each piece
      int piece = 0;
      sched::Walk w;
      for (w.start(share, p.kv_lens, p.Lk); w.valid(); w.next(p.kv_lens, p.Lk, units), ++piece) {
        ok = ptx::mbar_wait_a(BAR(kQEmpty), ((uint32_t)piece & 1u) ^ 1u, abort_flag, err,
                              kDevErrTimeoutProducer);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        if (lane == 0) {
          const int hkv = w.h / p.row_tiles, rt = w.h - hkv * p.row_tiles;
          const int rows_all = p.group * p.Lq;
          const int y = (w.b * p.Hkv + hkv) * rows_all + rt * 128;
          ptx::mbar_arrive_expect_tx(&bars[kQFull], C::kTileBytes);
          for (int a = 0; a < C::kAtoms; ++a)
            ptx::tma_load_2d(smem + C::kOffQ + a * C::kAtomBytes, &tm_q, &bars[kQFull], a * 64, y);
        }
        __syncwarp();
      }
      if (piece > 0 && lane == 0) {  // the last Q has landed
        int dummy = 0;
        ptx::mbar_wait_a(BAR(kQFull), (uint32_t)(piece - 1) & 1u, &dummy, nullptr, 0);
      }
    } else {
      // ------------------------------------------------------------ MMA issuer
      // S of tile j goes to buffer j % 2, two tiles ahead of its softmax; P lies over S,
      // so S of tile j + 2 follows tile j's P V in pipe order.
      constexpr uint32_t kIdescS = ptx::idesc_bf16_f32(128, 128, 0, 0);
      constexpr uint32_t kIdescPV = ptx::idesc_bf16_f32(128, D, 0, 1);
      const uint64_t q_desc = ptx::smem_desc_sw128(sq, 16, 1024);
      auto wait = [&](uint32_t bar, uint32_t parity) -> bool {
        const bool r = ptx::mbar_wait_a(bar, parity, abort_flag, err, kDevErrTimeoutMma);
        return __all_sync(0xffffffffu, r);
      };
      int base = 0;  // tiles of the earlier pieces
      int piece = 0;
      sched::Walk w;
      for (w.start(share, p.kv_lens, p.Lk); w.valid() && ok;
           w.next(p.kv_lens, p.Lk, units), ++piece) {
        const int end = base + w.t1 - w.t0;
        auto issue_s = [&](int j) -> bool {
          const int st = j % S;
          if (!wait(FULL(0, st), (uint32_t)(j / S) & 1u)) return false;
          ptx::tc_fence_after();
          const uint32_t s_tmem = tmem + (uint32_t)(j & 1) * 128u;
          const uint64_t k_desc = ptx::smem_desc_sw128(sk + st * C::kTileBytes, 16, 1024);
          if constexpr (D == 64)
            ptx::mma_qk_chain_d64(s_tmem, q_desc, k_desc, kIdescS);
          else
            ptx::mma_qk_chain_d128(s_tmem, q_desc, k_desc, kIdescS);
          ptx::mma_commit_warp(BAR(kSFull + (j & 1)));
          ptx::mma_commit_warp(EMPTY(0, st));
          if (j + 1 == end) ptx::mma_commit_warp(BAR(kQEmpty));
          return true;
        };
        ok = wait(BAR(kQFull), (uint32_t)piece & 1u) && issue_s(base);
        if (ok && base + 1 < end) ok = issue_s(base + 1);
        for (int j = base; j < end && ok; ++j) {
          const int st = j % S;
          const uint32_t s_tmem = tmem + (uint32_t)(j & 1) * 128u;
          const uint64_t v_desc =
              ptx::smem_desc_sw128(sv_ + st * C::kTileBytes, C::kAtomBytes, 1024);
          ok = wait(FULL(1, st), (uint32_t)(j / S) & 1u);
          if (ok && j == base && piece > 0)  // the previous piece's O have been read out
            ok = wait(BAR(kOFree), (uint32_t)(piece - 1) & 1u);
          for (int x = 0; x < 2 && ok; ++x) {
            ok = wait(BAR(kPFull + 2 * x + (j & 1)), (uint32_t)(j >> 1) & 1u);
            if (!ok) break;
            ptx::tc_fence_after();
            mma_pv_chain4(tmem + 256u + (uint32_t)(x * D), s_tmem + (uint32_t)(x * 64),
                          v_desc + (uint64_t)(x * 512), kIdescPV, j > base ? 1u : 0u);
            ptx::mma_commit_warp(BAR(kODone + 2 * x + (j & 1)));
          }
          if (!ok) break;
          ptx::mma_commit_warp(EMPTY(1, st));
          if (j + 1 == end) ptx::mma_commit_warp(BAR(kPieceDone));
          if (j + 2 < end) ok = issue_s(j + 2);
        }
        base = end;
      }
      ptx::mma_commit_warp(BAR(kDrain));
      int dummy = 0;
      ptx::mbar_wait_a(BAR(kDrain), 0, &dummy, nullptr, 0);
    }
  } else if (warp >= 12) {
    // ------------------------------------------------------------- expansion
    // A warpgroup per operand and half tile; warp w of it takes rows 16 w .. + 15; a
    // thread takes 16 codes of a row at a time, eight lanes on eight neighbouring rows
    // (conflict-free in both swizzled layouts).
    ptx::regs_dec<kRegsExpand>();
    constexpr int kH = D / 64;  // 16-code chunks per thread and row
    const int kv = (warp - 12) >> 3;
    const int half = (warp - 12) >> 2 & 1;  // of each tile
    const int row_w = (warp & 3) * 16 + (lane & 7);  // and + 8
    for (int j = 0; j < total; ++j) {
      const int st = j % S, fs = j % kFactorSlots;
      const uint32_t dst = (kv ? sv_ : sk) + st * C::kTileBytes;
      const uint8_t* factor = smem + C::kOffFactor + fs * 256 + kv * 128;
      const int hj = 2 * j + half, slot = hj % R;
      const uint32_t src = ptx::smem_u32(smem + C::kOffRaw + (kv * R + slot) * C::kRawBytes);
      ok = ptx::mbar_wait_a(BAR(kFactorFull + fs), (uint32_t)(j / kFactorSlots) & 1u, abort_flag,
                            err, kDevErrTimeoutProducer) &&
           ptx::mbar_wait_a(RAW_FULL(kv, slot), (uint32_t)(hj / R) & 1u, abort_flag, err,
                            kDevErrTimeoutProducer);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      // all loads first, so that they are in flight together
      uint32_t w[2][kH][4], f[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int r = row_w + 8 * i;
        f[i] = (uint32_t)factor[half * 64 + r] * 0x00800080u;
#pragma unroll
        for (int h = 0; h < kH; ++h) {
          const int q = (lane >> 3) + 4 * h;  // 16-code chunk of the row
          const uint32_t from = D == 128 ? (uint32_t)(r * 128 + ((q ^ (r & 7)) << 4))
                                         : (uint32_t)(r * 64 + ((q ^ ((r >> 1) & 3)) << 4));
          ptx::ld_shared_v4(src + from, w[i][h][0], w[i][h][1], w[i][h][2], w[i][h][3]);
        }
      }
      // a NaN code (magnitude 0x7f) carries into bit 7 of its byte; keys past the end (f = 0)
      // do not count
      uint32_t nan = 0;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        uint32_t x = 0;
#pragma unroll
        for (int h = 0; h < kH; ++h)
#pragma unroll
          for (int k = 0; k < 4; ++k) x |= (w[i][h][k] & 0x7f7f7f7fu) + 0x01010101u;
        nan |= f[i] != 0u ? x : 0u;
      }
      asm volatile(
          "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %0, 0;\n\t"
          "@p red.shared.max.u32 [%1], %2;\n\t}" ::"r"(nan & 0x80808080u),
          "r"(ptx::smem_u32(&misc->nan_end)), "r"(j + 1)
          : "memory");
      ok = ptx::mbar_wait_a(EMPTY(kv, st), ((uint32_t)(j / S) & 1u) ^ 1u, abort_flag, err,
                            kDevErrTimeoutProducer);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int r = half * 64 + row_w + 8 * i;
#pragma unroll
        for (int h = 0; h < kH; ++h) {
          const int q = (lane >> 3) + 4 * h;
          uint32_t o[8];
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            // bytes (b, sign b, b', sign b') of two neighbouring codes
            uint32_t x;
            asm("prmt.b32 %0, %1, 0, %2;"
                : "=r"(x)
                : "r"(w[i][h][k >> 1]), "r"(k & 1 ? 0xb3a2 : 0x9180));
            const uint32_t v = (x << 4) & 0x87f087f0u;
            const __nv_bfloat162 y = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&v),
                                             *reinterpret_cast<const __nv_bfloat162*>(&f[i]));
            o[k] = *reinterpret_cast<const uint32_t*>(&y);
          }
          // 16 values: chunks 2 (q % 4) and + 1 of atom q / 4
          const uint32_t row = dst + (uint32_t)((q >> 2) * C::kAtomBytes + r * 128);
          const int ch = (q & 3) * 2;
          asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(
                           row + (uint32_t)((ch ^ (r & 7)) << 4)),
                       "r"(o[0]), "r"(o[1]), "r"(o[2]), "r"(o[3])
                       : "memory");
          asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(
                           row + (uint32_t)(((ch + 1) ^ (r & 7)) << 4)),
                       "r"(o[4]), "r"(o[5]), "r"(o[6]), "r"(o[7])
                       : "memory");
        }
      }
      // the codes are in registers or stored: their slot may be loaded again
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive_a(RAW_EMPTY(kv, slot));
      ptx::fence_proxy_async_smem();
      ptx::mbar_arrive_a(FULL(kv, st));
      if (lane == 0) ptx::mbar_arrive_a(BAR(kFactorEmpty + fs));
    }
  } else {
    // ---------------------------------------------------------------- softmax
    ptx::regs_inc<kRegsSoftmax>();
    const int x = (warp - 4) >> 2;
    const int quarter = warp & 3;
    const int r = quarter * 32 + lane;  // row of the unit = TMEM lane
    const uint32_t t_row = tmem + ((uint32_t)(quarter * 32) << 16);
    const uint32_t o_col = 256u + (uint32_t)(x * D);
    float2* ml = reinterpret_cast<float2*>(smem + C::kOffMl);
    auto wait = [&](uint32_t bar, uint32_t parity) -> bool {
      const bool a = ptx::mbar_wait_a(bar, parity, abort_flag, err, kDevErrTimeoutSoftmax);
      return __all_sync(0xffffffffu, a);
    };
    int base = 0;  // tiles of the earlier pieces
    int piece = 0;
    sched::Walk w;
    for (w.start(share, p.kv_lens, p.Lk); w.valid() && ok;
         w.next(p.kv_lens, p.Lk, units), ++piece) {
      const int end = base + w.t1 - w.t0;
      const int key_end = min(w.t1 * 128, w.len);
      float m_ref = -INFINITY, l = 0.0f;
      for (int j = base; j < end; ++j) {
        // keys of this half tile below the end
        const int left = key_end - (w.t0 + j - base) * 128 - x * 64;
        ok = wait(BAR(kSFull + (j & 1)), (uint32_t)(j >> 1) & 1u);
        if (!ok) break;
        ptx::tc_fence_after();
        const float2 ref = misc->ref[j % kRefSlots];
        // not 0 where it underflows (keys of the smallest scales): -inf * 0 is NaN
        const float c = fmaxf(p.scale_log2 * ref.x, 0x1p-149f);
        const uint32_t s_col = t_row + (uint32_t)((j & 1) * 128 + x * 64);
        float s[64];
        {
          uint32_t r0[32], r1[32];
          ptx::tmem_ld32(s_col, r0);
          ptx::tmem_ld32(s_col + 32, r1);
          ptx::tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            s[i] = __uint_as_float(r0[i]);
            s[32 + i] = __uint_as_float(r1[i]);
          }
        }
        if (left < 64) {
#pragma unroll
          for (int i = 0; i < 64; ++i) s[i] = i < left ? s[i] : -INFINITY;
        }
        const float m_new = fmaxf(m_ref, row_max64(s) * c);
        const bool need = m_new > m_ref + kRescaleThreshold;
        const float alpha = need ? ptx::ex2(m_ref - m_new) : 1.0f;
        if (need) {
          l *= alpha;
          m_ref = m_new;
        }
        const float m_use = m_ref == -INFINITY ? 0.0f : m_ref;
        if (j > base && __any_sync(0xffffffffu, need)) {
          // O holds the P V of the piece's earlier tiles: final before it is rescaled
          ok = wait(BAR(kODone + 2 * x + ((j - 1) & 1)), (uint32_t)((j - 1) >> 1) & 1u);
          if (!ok) break;
          ptx::tc_fence_after();
#pragma unroll 1
          for (int cc = 0; cc < D / 32; ++cc) {
            uint32_t raw[32];
            ptx::tmem_ld32(t_row + o_col + cc * 32, raw);
            ptx::tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 32; ++i) raw[i] = __float_as_uint(__uint_as_float(raw[i]) * alpha);
            ptx::tmem_st32(t_row + o_col + cc * 32, raw);
          }
        }
        uint32_t pk[32];  // P' over this half of S
        const float sum = exp2_pack64(s, c, m_use - ref.y, pk);
        ptx::tmem_st32(s_col, pk);
        l += sum * ptx::ex2(-ref.y);
        ptx::tmem_wait_st();
        ptx::tc_fence_before();
        ptx::mbar_arrive_a(BAR(kPFull + 2 * x + (j & 1)));
      }
      if (!ok) break;
      // ------------------------------------------------------- end of the piece
      const int first = base;
      base = end;
      if (x == 1) {
        if (piece > 0) ok = wait(BAR(kMlEmpty), (uint32_t)(piece - 1) & 1u);
        if (!ok) break;
        ml[r] = make_float2(m_ref, l);
        ptx::mbar_arrive_a(BAR(kMlFull));
        continue;
      }
      ok = wait(BAR(kPieceDone), (uint32_t)piece & 1u) &&
           wait(BAR(kMlFull), (uint32_t)piece & 1u);
      if (!ok) break;
      ptx::tc_fence_after();
      const float2 other = ml[r];
      ptx::mbar_arrive_a(BAR(kMlEmpty));
      const int hkv = w.h / p.row_tiles, rt = w.h - hkv * p.row_tiles;
      uint32_t nan = 0;
      const uint32_t nan_end = *reinterpret_cast<volatile uint32_t*>(&misc->nan_end);
      if (__any_sync(0xffffffffu, nan_end > (uint32_t)first)) {
        nan = find_nan<D>(p, w.b, hkv, w.t0 * 128, key_end);
        if (nan >> 16) l = NAN;
      }
      const bool nan_cols = __any_sync(0xffffffffu, nan & 0xffffu);
      const float m = fmaxf(m_ref, other.x);
      const float mu = m == -INFINITY ? 0.0f : m;
      float a0 = ptx::ex2(m_ref - mu), a1 = ptx::ex2(other.x - mu);
      const float sum = a0 * l + a1 * other.y;
      const bool have = sum != 0.0f;  // NaN stays NaN
      const float inv = have ? 1.0f / sum : 0.0f;
      a0 *= inv;
      a1 *= inv;
      const float lse = have ? (mu + ptx::lg2(sum)) * kLn2 : -INFINITY;
      const int rows_all = p.group * p.Lq;
      const bool row_ok = r < rows_all - rt * 128;
      const bool final = w.whole();
      const long long row =
          final ? ((long long)w.b * p.Hkv + hkv) * rows_all + (long long)rt * 128 + r
                : (long long)w.slot(blockIdx.x) * 128 + r;
#pragma unroll 1
      for (int cc = 0; cc < D / 32; ++cc) {
        uint32_t e[32], o[32];
        ptx::tmem_ld32(t_row + 256u + cc * 32, e);
        ptx::tmem_ld32(t_row + 256u + D + cc * 32, o);
        ptx::tmem_wait_ld();
        if (nan_cols) {
          const uint32_t m = (__shfl_sync(0xffffffffu, nan, 2 * cc) & 0xffffu) |
                             __shfl_sync(0xffffffffu, nan, 2 * cc + 1) << 16;
#pragma unroll
          for (int i = 0; i < 32; ++i)
            if (m >> i & 1u) e[i] = 0x7fffffffu;
        }
        if (row_ok) {
          float v[32];
#pragma unroll
          for (int i = 0; i < 32; ++i)
            v[i] = a0 * __uint_as_float(e[i]) + a1 * __uint_as_float(o[i]);
          if (final) {
            __nv_bfloat16* dst = reinterpret_cast<__nv_bfloat16*>(p.o) + row * D + cc * 32;
#pragma unroll
            for (int i = 0; i < 32; i += 8)
              *reinterpret_cast<uint4*>(dst + i) = make_uint4(
                  ptx::pack_bf16x2(v[i], v[i + 1]), ptx::pack_bf16x2(v[i + 2], v[i + 3]),
                  ptx::pack_bf16x2(v[i + 4], v[i + 5]), ptx::pack_bf16x2(v[i + 6], v[i + 7]));
          } else {
            float* dst = p.ws_o + row * D + cc * 32;
#pragma unroll
            for (int i = 0; i < 32; i += 4)
              *reinterpret_cast<float4*>(dst + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
          }
        }
        __syncwarp();
      }
      if (row_ok) (final ? p.lse : p.ws_lse)[row] = lse;
      ptx::tc_fence_before();
      ptx::mbar_arrive_a(BAR(kOFree));
    }
  }

  // ------------------------------------------------------------------ teardown
  ptx::tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, kTmemCols);
  }
}

template <int D>
cudaError_t launch_decode_q8_wide(const CUtensorMap& tq, const CUtensorMap& tk,
                                  const CUtensorMap& tv, const DecodeParams& p,
                                  cudaStream_t stream) {
  auto kern = attn_decode_q8_wide_kernel<D>;
  constexpr int smem = WCfg<D>::kSmemAlloc;
  static PerContextOnce once;
  const cudaError_t e = once_per_context(once, [&](int) {
    return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  });
  if (e != cudaSuccess) return e;
  kern<<<p.num_ctas, kThreads, smem, stream>>>(tq, tk, tv, p);
  return cudaGetLastError();
}

template cudaError_t launch_decode_q8_wide<64>(const CUtensorMap&, const CUtensorMap&,
                                               const CUtensorMap&, const DecodeParams&,
                                               cudaStream_t);
template cudaError_t launch_decode_q8_wide<128>(const CUtensorMap&, const CUtensorMap&,
                                                const CUtensorMap&, const DecodeParams&,
                                                cudaStream_t);

}  // namespace attn
