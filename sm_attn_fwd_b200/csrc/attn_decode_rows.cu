// Split-KV decode with few query rows per KV head, over an 8-bit cache (format in
// cache_q8.cuh) or a bf16 one, for sm_100a.
//
//   S_ij = scale * <q_i, k_j>,   P = softmax(S),   O_i = sum_j P_ij v_j,
//   LSE_i = log sum_j exp(S_ij),   with k_j = 2^(ke_j - 127) kc_j and
//   v_j = 2^(ve_j - 127) vc_j for an 8-bit cache, whose codes kc, vc are never
//   expanded in memory.
//
// What bounds it is the stream of keys (2 (d + 1) or 4 d bytes per key and KV head for
// all query rows of the group), as long as turning them into matrix operands is
// cheap.  Few query rows share a key (8 at Lq = 1 with 8 heads per group), so the
// work is laid out around that: a warp owns whole keys and computes the
// transposed products with mma.m16n8k16 (fp32 out), whose N = 8 is the query rows
// and whose M = 16 is keys (S^T = K Q^T) or d (O^T = V^T P^T).  K and V go from
// shared memory to registers and are the A operand there (two instructions turn four
// codes into two f16 pairs, exactly): nothing is written back to shared memory,
// which the tcgen05 path would need for codes (its operands live in shared or tensor
// memory, and expanding 1 byte to 2 there moves 5 bytes of shared-memory traffic
// per code).
//
// Measured: 64 sequences x 8 KV heads, 32768 keys of d = 128 in 8 bits at most (2.7 GB),
// 8 query rows: 413 to 430 us, 6.3 to 6.5 TB/s, 96 to 99 % of the measured copy
// bandwidth.  At d = 64 a key has half the bytes and as many instructions but for its
// products: 16 x 16 heads x 16384 keys take 115 to 120 us, 4.5 to 4.7 TB/s, with 58 % of
// the issue slots and 55 % of the integer pipe (conversions, permutes) in use.  16 x 16
// heads of up to 4099 keys: 27 to 29 us against 10.4 at the copy bandwidth, where the start, the
// pieces' ends and the merge kernel are about half of the time.
//
// Numbers, 8-bit cache.  Q is scaled per row by a power of two into f16's upper range
// (an element keeps all 8 bits of its bf16 significand down to 2^-31 of the row's
// largest).  Scores, maxima and sums are fp32.  P times the value scale goes into
// the second product as f16 relative to a running reference of its own, R_i between
// w_i - 15 and w_i - 7, w_i = max_j (S_ij log2 e + ve_j), separate from the softmax's
// reference m_i: a value row with a large scale but a small weight then costs the others
// nothing.  f16 rounds P to 11 bits, 8 times finer than bf16, and its largest P is 2^7
// to 2^15, so that half its smallest step, what a key with next to no weight may lose, is
// at most 2^-32 of the row's largest P 2^ve.  (Most keys of a long context are such keys:
// with R_i = w_i a flat tail of weights below 2^-25 vanished, however long.)  bf16 cache:
// both products take bf16 as it is, P rounded to it, and R_i = m_i.
//
// Layout of a warp's block (32 keys; 16 for bf16 at d = 128) in groups of 16 keys.  A
// contraction does not care about the order of its terms, so d and the keys are
// permuted to let every thread read 16 consecutive bytes (8 for V codes at d = 64):
//   S^T: thread (g = lane / 4, t = lane % 4) reads 16-byte chunks t, t + 4, ... of
//     keys sigma(g) and 8 + sigma(g); a chunk of codes is 4 k-steps, of bf16 2.
//   O^T: it reads its part of d (codes: d / 8 bytes from (d / 8) g; bf16: chunk g of
//     each 64 columns) of keys sigma(2t), sigma(2t + 1), + 8; a byte permute of two
//     keys' words pairs the keys, as the operand wants.
// sigma (a permutation of 0..7) makes both reads conflict-free in the swizzled
// tile; P^T comes from S^T by movmatrix (8x8 transposes), with no shared memory.
//
// Every warp streams its own blocks through its own ring (TMA boxes, one mbarrier per
// stage; lane 0 issues), so warps wait for one another only where a piece of work
// (decode_sched.cuh) ends and their results are merged; with 16-key pages as many
// lanes issue boxes as there are warps.  The ring runs on across pieces.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "attn_params.h"
#include "cache_q8.cuh"
#include "decode_params.h"
#include "host_once.h"
#include "ptx.cuh"
#include "decode_sched.cuh"

namespace attn {
namespace {

constexpr float kSlack = 8.0f;        // log2 units a running reference may lag behind
// 8-bit cache: how far R lies below the largest P 2^ve, in log2 units.  With the lag P
// stays at or below 2^15, inside f16's range.
constexpr float kHeadroom = 7.0f;
constexpr float kLn2 = 0.69314718055994530942f;
// The running references before the first score: finite, so that a block whose scores
// all overflow to -inf adds 2^(-inf) = 0, not 2^(-inf + inf).
constexpr float kLowest = -3.0e38f;

// Warps per CTA (one CTA per SM): as many as the registers allow, since a warp's
// chain of dependent steps per block, not the issue rate, is what more warps hide.
template <int D, int NB, bool kQ8>
struct RowCfg {
  static constexpr int kWarps =
      NB == 4 || (NB == 2 && D == 128) ? 8 : kQ8 && D == 64 && NB == 1 ? 16 : 12;
  static constexpr int kThreads = kWarps * 32;
  static constexpr int kRows = 8 * NB;                       // query rows per unit
  static constexpr int kUnit = !kQ8 && D == 128 ? 16 : 32;   // keys a warp takes at a time
  static constexpr int kAtoms = kQ8 ? 1 : D / 64;            // swizzled columns of a tile
  static constexpr int kRowBytes = kQ8 ? D : 128;            // of one key in one of them
  static constexpr int kAtomBytes = kUnit * kRowBytes;
  static constexpr int kTileBytes = kAtoms * kAtomBytes;     // one K or V block
  static constexpr int kStageBytes = 2 * kTileBytes;
  static constexpr int kStages = kQ8 && D == 64 ? (NB == 4 ? 4 : 3) : 2;
  static constexpr int kRingBytes = kWarps * kStages * kStageBytes;
  // merge buffers: a warp's accumulators and statistics, one 128-byte row per register
  static constexpr int kMergeRegs = NB * (D / 16 * 4 + 6);
  static constexpr int kMergeBufs = kWarps == 12 ? 4 : kWarps / 2;
  static constexpr int kMergeBytes = kMergeBufs * kMergeRegs * 128;
  static constexpr int kOffMerge = kRingBytes;
  static constexpr int kOffExp = kOffMerge + kMergeBytes;  // [warp][stage][K, V][32] scale bytes
  static constexpr int kOffQ = kOffExp + (kQ8 ? kWarps * kStages * 64 : 0);  // Q of two pieces
  static constexpr int kOffBar = kOffQ + 2 * kRows * D * 2;
  static constexpr int kOffMisc = kOffBar + (kWarps * kStages + 2) * 8;
  static constexpr int kSmemBytes = kOffMisc + 64;
  static constexpr int kSmemAlloc = kSmemBytes + 1024;  // slack for 1024-byte alignment
  static_assert(kSmemAlloc <= 227 * 1024, "shared memory");
};

// Returns once the kernel before this one in the stream is complete and its writes
// are visible (this one may have started earlier).
__device__ __forceinline__ void wait_for_previous_kernel() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

// Key of mma row g inside its group of 8 (see the head of this file).
//   128-byte rows: sigma(2t + 1) = sigma(2t) ^ 4, and sigma(2t) >> 1 = t;
//   64-byte rows: sigma(2t + 1) = sigma(2t) ^ 3, sigma(2t) in {0, 1, 4, 5}.
template <int kRowBytes>
__device__ __forceinline__ int sigma(int g) {
  if constexpr (kRowBytes == 128) return ((g & 6) + (g >> 2)) ^ ((g & 1) << 2);
  return (((g >> 1) & 1) | (g & 4)) ^ (g & 1 ? 3 : 0);
}

// Byte offset of 16-byte chunk c of key row r in a unit as TMA lays it out
// (128-byte swizzle for 128-byte rows, 64-byte swizzle for 64-byte rows).
template <int kRowBytes>
__device__ __forceinline__ uint32_t chunk_off(int r, int c) {
  if constexpr (kRowBytes == 128) return (uint32_t)(r * 128 + ((c ^ (r & 7)) << 4));
  return (uint32_t)(r * 64 + ((c ^ ((r >> 1) & 3)) << 4));
}

template <bool kF16>
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  if constexpr (kF16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// A copy of `bytes` (a multiple of 16) from global to shared memory, both 16-byte
// aligned, counted on the mbarrier.
__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes,
                                          uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::
          "r"(ptx::smem_u32(dst)),
      "l"(src), "r"(bytes), "r"(ptx::smem_u32(bar))
      : "memory");
}

__device__ __forceinline__ void ld_shared_v2(uint32_t addr, uint32_t& a, uint32_t& b) {
  asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(a), "=r"(b) : "r"(addr));
}

}  // namespace

template <int D, int NB, bool kQ8>
__global__ void __launch_bounds__(RowCfg<D, NB, kQ8>::kThreads, 1)
    attn_decode_rows_kernel(const __grid_constant__ CUtensorMap tm_k,
                          const __grid_constant__ CUtensorMap tm_v, const DecodeParams p) {
  using C = RowCfg<D, NB, kQ8>;
  constexpr int S = C::kStages;
  constexpr int kWarps = C::kWarps;
  constexpr int kUnit = C::kUnit;
  constexpr int kSub = kUnit / 16;   // 16-key groups of a block
  constexpr int kRB = C::kRowBytes;
  constexpr int kMu = D / 16;  // M tiles of O^T
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  const int units = p.Hkv * p.row_tiles;

  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::kOffBar) + warp * S;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::kOffMisc);
  sched::Share* share = reinterpret_cast<sched::Share*>(smem + C::kOffMisc + 8);
  if (lane == 0) {
    for (int s = 0; s < S; ++s) ptx::mbar_init(&bars[s], 1);
    ptx::fence_mbar_init();
  }
  uint64_t* q_bars = reinterpret_cast<uint64_t*>(smem + C::kOffBar) + kWarps * S;
  if (warp == 0) {
    if (lane == 0) {
      ptx::mbar_init(&q_bars[0], 1);
      ptx::mbar_init(&q_bars[1], 1);
      ptx::fence_mbar_init();
    }
    const sched::Share sh =
        sched::find_share(p.kv_lens, p.B, p.Lk, units, p.piece, blockIdx.x, gridDim.x, p.err);
    if (lane == 0) {
      *share = sh;
      *abort_flag = 0;
    }
  } else if (threadIdx.x == 32) {
    ptx::prefetch_tmap(&tm_k);
    ptx::prefetch_tmap(&tm_v);
  }
  __syncthreads();
  sched::let_next_kernel_launch();

  // Q of a piece, one copy of its rows (they lie one after another) into buffer
  // piece % 2, by one thread a piece ahead.
  const int rows_all = p.group * p.Lq;
  int q_issued = 0;
  auto load_q = [&](const sched::Walk& a, int piece) {
    const int hkv = a.h / p.row_tiles, rt = a.h - hkv * p.row_tiles;
    const long long row = ((long long)a.b * p.Hkv + hkv) * rows_all + (long long)rt * C::kRows;
    const uint32_t bytes = (uint32_t)(min(C::kRows, rows_all - rt * C::kRows) * D * 2);
    ptx::mbar_arrive_expect_tx(&q_bars[piece & 1], bytes);
    bulk_load(smem + C::kOffQ + (piece & 1) * (C::kRows * D * 2),
              reinterpret_cast<const __nv_bfloat16*>(p.q) + row * D, bytes, &q_bars[piece & 1]);
    q_issued = piece + 1;
  };

  // ------------------------------------------------------------------ loads
  uint8_t* ring = smem + warp * S * C::kStageBytes;
  uint8_t* exps = smem + C::kOffExp + warp * S * 64;
  const bool paged = p.block_table != nullptr;
  const uint64_t kv_policy = ptx::l2_policy_evict_first();
  // The block this warp loads next: keys [l_key, l_end) of piece `lw` hold it and the
  // warp's later ones; z: pool index (page * Hkv + hkv) of the page of this lane's key,
  // -1 past the end or for a page id outside the pool (reads as zeros).
  sched::Walk lw;
  lw.start(*share, p.kv_lens, p.Lk);
  int l_key = 0, l_end = 0, z = -1;
  auto find_block = [&]() {  // move to a piece with a block for this warp, and fetch its page
    while (lw.valid() && l_key >= l_end) {
      lw.next(p.kv_lens, p.Lk, units);
      l_key = lw.t0 * 128 + warp * kUnit;
      l_end = min(lw.t1 * 128, lw.len);
    }
    if (!lw.valid()) return;
    const int hkv = lw.h / p.row_tiles;
    z = lw.b * p.Hkv + hkv;
    if (paged) {
      z = -1;
      const int j = l_key + lane;
      if (lane < kUnit && j < l_end) {
        const int page = __ldg(p.block_table + (long long)lw.b * p.pages_per_seq +
                               (j >> p.page_shift));
        if (page >= 0 && page < p.num_pages)
          z = page * p.Hkv + hkv;
        else
          atomicOr(p.err, kDevErrBadPage);
      }
    }
  };
  l_key = lw.t0 * 128 + warp * kUnit;
  l_end = min(lw.t1 * 128, lw.len);
  find_block();
  int n_issued = 0;
  // the scale bytes of block i
  auto store_exps = [&](int i, int ke, int ve) {
    uint8_t* dst = exps + i % S * 64;
    dst[lane] = (uint8_t)min(ke, q8::kMaxScaleByte);
    dst[32 + lane] = (uint8_t)min(ve, q8::kMaxScaleByte);
  };
  // Issue the boxes of the next block (one per operand, or one per page slice for pages
  // shorter than a block), load its scale bytes and find the block after it.
  auto issue = [&](int& ke, int& ve) {
    const int s = n_issued % S;
    uint8_t* kd = ring + s * C::kStageBytes;
    uint8_t* vd = kd + C::kTileBytes;
    if (lane == 0) ptx::mbar_arrive_expect_tx(&bars[s], C::kStageBytes);
    __syncwarp();
    const int rows = paged ? min(p.page_size, kUnit) : kUnit;
    if (lane < kUnit && (lane & (rows - 1)) == 0) {
      const int j = l_key + lane;
      const int y = paged ? j & (p.page_size - 1) : j;
#pragma unroll
      for (int a = 0; a < C::kAtoms; ++a) {
        const int off = a * C::kAtomBytes + lane * kRB;
        ptx::tma_load_3d_hint(kd + off, &tm_k, &bars[s], a * 64, y, z, kv_policy);
        ptx::tma_load_3d_hint(vd + off, &tm_v, &bars[s], a * 64, y, z, kv_policy);
      }
    }
    ke = ve = 1;
    const int j = l_key + lane;
    if (kQ8 && j < l_end && z >= 0) {
      const long long at = paged ? ((long long)z << p.page_shift) + (j & (p.page_size - 1))
                                 : (long long)z * p.Lk + j;
      ke = __ldg(p.k_exp + at);
      ve = __ldg(p.v_exp + at);
    }
    ++n_issued;
    l_key += kWarps * kUnit;
    find_block();
  };
  {
    int ke[S], ve[S];  // every load goes out before the first is waited for
#pragma unroll
    for (int i = 0; i < S; ++i)
      if (lw.valid()) issue(ke[i], ve[i]);
#pragma unroll
    for (int i = 0; i < S; ++i)
      if (kQ8 && i < n_issued) store_exps(i, ke[i], ve[i]);
  }
  int pend_ke = 1, pend_ve = 1;  // scale bytes of the block issued last
  bool pending = false;          // not stored yet

  const int sg = sigma<kRB>(g), s2t0 = sigma<kRB>(2 * t), s2t1 = sigma<kRB>(2 * t + 1);
  bool ok = true;
  int done = 0;  // blocks consumed
  float* merge = reinterpret_cast<float*>(smem + C::kOffMerge);
  sched::Walk w;
  w.start(*share, p.kv_lens, p.Lk);
  if (threadIdx.x == 0 && w.valid()) load_q(w, 0);
  for (int piece = 0; w.valid(); ++piece) {
    sched::Walk next = w;  // the piece after this one
    next.next(p.kv_lens, p.Lk, units);
    if (threadIdx.x == 0 && next.valid()) load_q(next, piece + 1);
    const int hkv = w.h / p.row_tiles, rt = w.h - hkv * p.row_tiles;
    const int rows_valid = min(C::kRows, rows_all - rt * C::kRows);
    // flat output row of the unit's first row
    const long long row0 =
        ((long long)w.b * p.Hkv + hkv) * rows_all + (long long)rt * C::kRows;
    const int key_end = min(w.t1 * 128, w.len);

    // ----------------------------------------------------------------- Q
    // B operand of S^T: query row n = g of each 8-row block, d in the order above
    uint32_t qf[NB][D / 16][2];
    float fac0[NB], fac1[NB];  // scale * log2 e * 2^(row shift) of query rows 2t and 2t + 1
    ok = ok && ptx::mbar_wait_a(ptx::smem_u32(&q_bars[piece & 1]), (uint32_t)(piece >> 1) & 1u,
                                abort_flag, p.err, kDevErrTimeoutProducer);
    const uint4* q_s =
        reinterpret_cast<const uint4*>(smem + C::kOffQ + (piece & 1) * (C::kRows * D * 2));
    if constexpr (!kQ8) {
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        const int r = nb * 8 + g;
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {  // chunks t, t + 4, ...: two k-steps each
          const uint4 x =
              r < rows_valid ? q_s[r * (D / 8) + c * 4 + t] : make_uint4(0, 0, 0, 0);
          qf[nb][2 * c][0] = x.x;
          qf[nb][2 * c][1] = x.y;
          qf[nb][2 * c + 1][0] = x.z;
          qf[nb][2 * c + 1][1] = x.w;
        }
        fac0[nb] = fac1[nb] = p.scale_log2;
      }
    } else {
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        uint4 raw[(D / 64)][2];
        const int r = nb * 8 + g;
#pragma unroll
        for (int j = 0; j < (D / 64); ++j)
#pragma unroll
          for (int h = 0; h < 2; ++h)
            raw[j][h] =
                r < rows_valid ? q_s[r * (D / 8) + j * 8 + t * 2 + h] : make_uint4(0, 0, 0, 0);
        float amax = 0.0f;
#pragma unroll
        for (int j = 0; j < (D / 64); ++j)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint32_t x[4] = {raw[j][h].x, raw[j][h].y, raw[j][h].z, raw[j][h].w};
#pragma unroll
            for (int i = 0; i < 4; ++i)
              amax = fmaxf(amax, fmaxf(fabsf(__uint_as_float(x[i] << 16)),
                                       fabsf(__uint_as_float(x[i] & 0xffff0000u))));
          }
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
        // the row times 2^(14 - exponent of amax), so that its largest lies in [2^14, 2^15);
        // in two factors, as 2^(14 + 126) is no fp32 number
        const int ex = max((int)(__float_as_uint(amax) >> 23), 1) - 127;
        const int sh = 14 - ex;
        const float s1 = __uint_as_float((uint32_t)(127 + sh / 2) << 23);
        const float s2 = __uint_as_float((uint32_t)(127 + sh - sh / 2) << 23);
#pragma unroll
        for (int j = 0; j < (D / 64); ++j)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint32_t x[4] = {raw[j][h].x, raw[j][h].y, raw[j][h].z, raw[j][h].w};
#pragma unroll
            for (int i = 0; i < 4; ++i)
              qf[nb][j * 4 + h * 2 + (i >> 1)][i & 1] =
                  pack_f16x2(__uint_as_float(x[i] << 16) * s1 * s2,
                             __uint_as_float(x[i] & 0xffff0000u) * s1 * s2);
          }
        // rows 2t and 2t + 1 live in lanes 8t and 8t + 4
        const int sh0 = __shfl_sync(0xffffffffu, sh, 8 * t);
        const int sh1 = __shfl_sync(0xffffffffu, sh, 8 * t + 4);
        fac0[nb] = p.scale_log2 * __uint_as_float((uint32_t)(127 - sh0 / 2) << 23) *
                   __uint_as_float((uint32_t)(127 - (sh0 - sh0 / 2)) << 23);
        fac1[nb] = p.scale_log2 * __uint_as_float((uint32_t)(127 - sh1 / 2) << 23) *
                   __uint_as_float((uint32_t)(127 - (sh1 - sh1 / 2)) << 23);
      }
    }

    // ------------------------------------------------------------- key blocks
    float o[NB][kMu][4];
    float m[NB][2], R[NB][2], l[NB][2];
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
      for (int mu = 0; mu < kMu; ++mu)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[nb][mu][i] = 0.0f;
      m[nb][0] = m[nb][1] = R[nb][0] = R[nb][1] = kLowest;
      l[nb][0] = l[nb][1] = 0.0f;
    }
    for (int k0 = w.t0 * 128 + warp * kUnit; k0 < key_end; k0 += kWarps * kUnit) {
      const int s = done % S;
      const int left = key_end - k0;  // visible keys of the block: [0, left)
      // lanes may give up a wait apart from each other (that for Q too), and the votes below
      // need them all: only this one ends the loop
      ok = ok && ptx::mbar_wait_a(ptx::smem_u32(&bars[s]), (uint32_t)(done / S) & 1u, abort_flag,
                                  p.err, kDevErrTimeoutProducer);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      if (kQ8 && pending) store_exps(n_issued - 1, pend_ke, pend_ve);
      __syncwarp();
      const uint32_t sk = ptx::smem_u32(ring + s * C::kStageBytes);
      const uint32_t sv = sk + C::kTileBytes;
      [[maybe_unused]] const uint8_t* eb = exps + s * 64;

      // S^T of the 16-key groups
      float z[kSub][NB][4];
#pragma unroll
      for (int blk = 0; blk < kSub; ++blk) {
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int i = 0; i < 4; ++i) z[blk][nb][i] = 0.0f;
        // 16-byte chunks of the keys: atom c / 2 (bf16), chunk t or t + 4 of it
        constexpr int kChunks = kQ8 ? D / 64 : D / 32;
#pragma unroll
        for (int c = 0; c < kChunks; ++c) {
          const uint32_t at = sk + (kQ8 ? 0 : (c >> 1) * C::kAtomBytes);
          const int ch = (kQ8 ? c * 4 : (c & 1) * 4) + t;
          uint32_t wa[4], wb[4];
          ptx::ld_shared_v4(at + chunk_off<kRB>(blk * 16 + sg, ch), wa[0], wa[1], wa[2], wa[3]);
          ptx::ld_shared_v4(at + chunk_off<kRB>(blk * 16 + 8 + sg, ch), wb[0], wb[1], wb[2],
                            wb[3]);
          if constexpr (kQ8) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              uint32_t a0, a1, a2, a3;
              q8::codes4_to_f16(wa[i], a0, a2);
              q8::codes4_to_f16(wb[i], a1, a3);
#pragma unroll
              for (int nb = 0; nb < NB; ++nb)
                mma16816<true>(z[blk][nb], a0, a1, a2, a3, qf[nb][c * 4 + i][0],
                               qf[nb][c * 4 + i][1]);
            }
          } else {
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
              for (int nb = 0; nb < NB; ++nb)
                mma16816<false>(z[blk][nb], wa[2 * h], wb[2 * h], wa[2 * h + 1], wb[2 * h + 1],
                                qf[nb][c * 2 + h][0], qf[nb][c * 2 + h][1]);
          }
        }
      }
      // scores in the base-2 domain; z[..][i]: key blk * 16 + (i / 2) * 8 + sigma(g), row
      // 2t + i % 2
      float vexp[kSub][2];
#pragma unroll
      for (int blk = 0; blk < kSub; ++blk)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int key = blk * 16 + h * 8 + sg;
          float ks = 1.0f;
          if constexpr (kQ8) {
            ks = q8::scale_of(eb[key]);
            vexp[blk][h] = (float)((int)eb[32 + key] - 127);
          }
          const bool vis = key < left;
#pragma unroll
          for (int nb = 0; nb < NB; ++nb) {
            z[blk][nb][2 * h] = vis ? z[blk][nb][2 * h] * (ks * fac0[nb]) : -INFINITY;
            z[blk][nb][2 * h + 1] = vis ? z[blk][nb][2 * h + 1] * (ks * fac1[nb]) : -INFINITY;
          }
        }
      // the thread's largest score of row 2t + i, and largest score times value scale
      auto max_z = [&](int nb, int i) {
        float v = -INFINITY;
#pragma unroll
        for (int blk = 0; blk < kSub; ++blk)
          v = fmaxf(v, fmaxf(z[blk][nb][i], z[blk][nb][2 + i]));
        return v;
      };
      auto max_w = [&](int nb, int i) {
        float v = -INFINITY;
#pragma unroll
        for (int blk = 0; blk < kSub; ++blk)
          v = fmaxf(v, fmaxf(z[blk][nb][i] + vexp[blk][0], z[blk][nb][2 + i] + vexp[blk][1]));
        return v;
      };
      // running references: raised only when a score passes one by more than kSlack
      bool need = false;
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          need |= max_z(nb, i) > m[nb][i] + kSlack;
          // (a difference, as a sum is rounded where scores are large, and P must not pass 2^15)
          if constexpr (kQ8) need |= max_w(nb, i) - R[nb][i] > kSlack + kHeadroom;
        }
      if (__any_sync(0xffffffffu, need)) {
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            float zm = max_z(nb, i), wm = kQ8 ? max_w(nb, i) : 0.0f;
#pragma unroll
            for (int x = 4; x < 32; x <<= 1) {
              zm = fmaxf(zm, __shfl_xor_sync(0xffffffffu, zm, x));
              if constexpr (kQ8) wm = fmaxf(wm, __shfl_xor_sync(0xffffffffu, wm, x));
            }
            wm = kQ8 ? wm - kHeadroom : zm;
            if (zm > m[nb][i]) {
              l[nb][i] *= ptx::ex2(m[nb][i] - zm);
              m[nb][i] = zm;
            }
            if (wm > R[nb][i]) {
              const float a = ptx::ex2(R[nb][i] - wm);
              R[nb][i] = wm;
#pragma unroll
              for (int mu = 0; mu < kMu; ++mu) {
                o[nb][mu][i] *= a;
                o[nb][mu][2 + i] *= a;
              }
            }
          }
      }
      // row sums and P^T (times the value scales) as the B operand of O^T
      uint32_t pb[kSub][NB][2];
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int blk = 0; blk < kSub; ++blk)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const float z0 = z[blk][nb][2 * h], z1 = z[blk][nb][2 * h + 1];
            const float p0 = ptx::ex2(z0 - m[nb][0]), p1 = ptx::ex2(z1 - m[nb][1]);
            l[nb][0] += p0;
            l[nb][1] += p1;
            if constexpr (kQ8) {
              const float w0 = ptx::ex2(z0 + vexp[blk][h] - R[nb][0]);
              const float w1 = ptx::ex2(z1 + vexp[blk][h] - R[nb][1]);
              pb[blk][nb][h] = transpose8x8(pack_f16x2(w0, w1));
            } else {
              pb[blk][nb][h] = transpose8x8(ptx::pack_bf16x2(p0, p1));
            }
          }
      // O^T += V^T P^T
#pragma unroll
      for (int blk = 0; blk < kSub; ++blk)
#pragma unroll
        for (int a = 0; a < C::kAtoms; ++a) {
          constexpr int kW = kQ8 ? D / 32 : 4;  // words per thread and key
          uint32_t vw[4][kW];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int key = blk * 16 + (i & 1 ? s2t1 : s2t0) + (i >> 1) * 8;
            const uint32_t at = sv + a * C::kAtomBytes;
            if constexpr (kW == 4)
              ptx::ld_shared_v4(at + chunk_off<kRB>(key, g), vw[i][0], vw[i][1], vw[i][2],
                                vw[i][3]);
            else
              ld_shared_v2(at + chunk_off<kRB>(key, g >> 1) + (g & 1) * 8, vw[i][0], vw[i][1]);
            // a masked key's values may be anything (even NaN): 0 * NaN would poison O
            if (left < kUnit && key >= left) {
#pragma unroll
              for (int x = 0; x < kW; ++x) vw[i][x] = 0u;
            }
          }
#pragma unroll
          for (int x = 0; x < kW; ++x) {
            if constexpr (kQ8) {
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                const uint32_t sel = h ? 0x7362 : 0x5140;  // bytes 2h, 2h + 1 of two keys
                uint32_t a0, a1, a2, a3;
                q8::codes4_to_f16(__byte_perm(vw[0][x], vw[1][x], sel), a0, a1);
                q8::codes4_to_f16(__byte_perm(vw[2][x], vw[3][x], sel), a2, a3);
#pragma unroll
                for (int nb = 0; nb < NB; ++nb)
                  mma16816<true>(o[nb][2 * x + h], a0, a1, a2, a3, pb[blk][nb][0],
                                 pb[blk][nb][1]);
              }
            } else {
              const uint32_t a0 = __byte_perm(vw[0][x], vw[1][x], 0x5410);
              const uint32_t a1 = __byte_perm(vw[0][x], vw[1][x], 0x7632);
              const uint32_t a2 = __byte_perm(vw[2][x], vw[3][x], 0x5410);
              const uint32_t a3 = __byte_perm(vw[2][x], vw[3][x], 0x7632);
#pragma unroll
              for (int nb = 0; nb < NB; ++nb)
                mma16816<false>(o[nb][a * 4 + x], a0, a1, a2, a3, pb[blk][nb][0],
                                pb[blk][nb][1]);
            }
          }
        }
      // every lane has read the stage: the next block may land there
      __syncwarp();
      ++done;
      pending = lw.valid();
      if (pending) issue(pend_ke, pend_ve);
    }

    // ----------------------------------------------------------------- merge
    // Warps leave O (in units of 2^R), m, R and their lanes' parts of l in shared memory,
    // one 128-byte row per register.  While there are more warps than buffers, the last
    // ones' results are added to the first ones'; then all threads merge the rest
    // and write the result.  Only warps that had a block of the piece take part.
    auto leave = [&](int buf) {
      float* dst = merge + buf * (C::kMergeRegs * 32) + lane;
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          dst[(nb * 6 + i) * 32] = m[nb][i];
          dst[(nb * 6 + 2 + i) * 32] = R[nb][i];
          dst[(nb * 6 + 4 + i) * 32] = l[nb][i];
        }
#pragma unroll
        for (int mu = 0; mu < kMu; ++mu)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            dst[(NB * 6 + (nb * kMu + mu) * 4 + i) * 32] = o[nb][mu][i];
      }
    };
    ok = __syncthreads_and(ok ? 1 : 0) != 0;  // also: the buffers are free again
    const int blocks = (key_end - w.t0 * 128 + kUnit - 1) / kUnit;
    int n = min(kWarps, blocks);
    while (n > C::kMergeBufs) {
      const int keep = max(n - C::kMergeBufs, C::kMergeBufs);
      if (warp >= keep && warp < n) leave(warp - keep);
      __syncthreads();
      if (warp < n - keep) {
        const float* src = merge + warp * (C::kMergeRegs * 32) + lane;
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          float a0[2], a1[2];  // weights of this warp's and the other's O
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float m1 = src[(nb * 6 + i) * 32], R1 = src[(nb * 6 + 2 + i) * 32];
            const float mn = fmaxf(m[nb][i], m1), Rn = fmaxf(R[nb][i], R1);
            l[nb][i] = l[nb][i] * ptx::ex2(m[nb][i] - mn) +
                       src[(nb * 6 + 4 + i) * 32] * ptx::ex2(m1 - mn);
            a0[i] = ptx::ex2(R[nb][i] - Rn);
            a1[i] = ptx::ex2(R1 - Rn);
            m[nb][i] = mn;
            R[nb][i] = Rn;
          }
#pragma unroll
          for (int mu = 0; mu < kMu; ++mu)
#pragma unroll
            for (int i = 0; i < 4; ++i)
              o[nb][mu][i] = o[nb][mu][i] * a0[i & 1] +
                             src[(NB * 6 + (nb * kMu + mu) * 4 + i) * 32] * a1[i & 1];
        }
      }
      n = keep;
      __syncthreads();
    }
    if (warp < n) leave(warp);
    __syncthreads();
    const bool final = w.whole();
    const long long at = final ? row0 : (long long)w.slot(blockIdx.x) * C::kRows;
    // a warp's item: two consecutive d of rows 2t + i, i.e. registers (nb, mu, i) and
    // (nb, mu, 2 + i) of every lane
    for (int item = warp; item < NB * 2 * kMu; item += kWarps) {
      const int nb = item / (2 * kMu), i = item / kMu & 1, mu = item % kMu;
      const float* st = merge + (nb * 6 + i) * 32 + lane;
      const float* ov = merge + (NB * 6 + (nb * kMu + mu) * 4 + i) * 32 + lane;
      float M = kLowest, Rm = kLowest;
#pragma unroll
      for (int x = 0; x < C::kMergeBufs; ++x)
        if (x < n) {
          M = fmaxf(M, st[x * C::kMergeRegs * 32]);
          Rm = fmaxf(Rm, st[x * C::kMergeRegs * 32 + 64]);
        }
      float ls = 0.0f, v0 = 0.0f, v1 = 0.0f;
#pragma unroll
      for (int x = 0; x < C::kMergeBufs; ++x)
        if (x < n) {
          const int off = x * C::kMergeRegs * 32;
          ls += st[off + 128] * ptx::ex2(st[off] - M);
          const float a = ptx::ex2(st[off + 64] - Rm);
          v0 += a * ov[off];
          v1 += a * ov[off + 64];
        }
#pragma unroll
      for (int x = 4; x < 32; x <<= 1) ls += __shfl_xor_sync(0xffffffffu, ls, x);
      const bool have = ok && ls != 0.0f;  // NaN stays NaN
      const float inv = have ? 1.0f / ls : 0.0f;
      // O is in units of 2^R, l in units of 2^m.  In two factors: with the smallest value
      // scales 2^(R - m) is no normal number, and ex2 would give 0.
      const float f = ptx::ex2(0.5f * (Rm - M));
      v0 = v0 * inv * f * f;
      v1 = v1 * inv * f * f;
      const int r = nb * 8 + 2 * t + i;
      if (r < rows_valid) {
        const int col = kQ8 ? g * (D / 8) + 2 * mu : (mu >> 2) * 64 + g * 8 + 2 * (mu & 3);
        const long long to = (at + r) * D + col;
        if (final && !p.own_o)
          *reinterpret_cast<uint32_t*>(reinterpret_cast<__nv_bfloat16*>(p.o) + to) =
              ptx::pack_bf16x2(v0, v1);
        else
          *reinterpret_cast<float2*>((final ? p.own_o : p.ws_o) + to) = make_float2(v0, v1);
        if (mu == 0 && g == 0)
          (!final ? p.ws_lse : p.own_o ? p.own_lse : p.lse)[at + r] = have ? (M + ptx::lg2(ls)) * kLn2 : -INFINITY;
      }
    }
    if (!ok) break;
    w = next;
  }
  // Where this kernel started before the one ahead of it had ended, it ends after it, so
  // that the merge that waits for this one has both.
  wait_for_previous_kernel();
  if (!ok && threadIdx.x == 0) {
    for (int i = max(0, q_issued - 2); i < q_issued; ++i) {
      int dummy = 0;
      ptx::mbar_wait_a(ptx::smem_u32(&q_bars[i & 1]), (uint32_t)(i >> 1) & 1u, &dummy, nullptr, 0);
    }
  }
  if (!ok && lane == 0) {
    // a wait gave up: let the copies in flight land before the CTA goes away
    for (int i = done; i < n_issued; ++i) {
      int dummy = 0;
      ptx::mbar_wait_a(ptx::smem_u32(&bars[i % S]), (uint32_t)(i / S) & 1u, &dummy, nullptr, 0);
    }
  }
}

// Merges the pieces of units that several CTAs computed, and the partial results of
// num_prefix splits of a shared prefix where there are any,
//   LSE = log sum_s exp(LSE_s),  O = sum_s exp(LSE_s - LSE) O_s,
// and writes the empty result of sequences without keys.  One warp per output row;
// lane i owns d / 32 consecutive elements.
//
// kBatch results' rows are in flight together, the first ones with their LSEs.  With few
// output rows a batch costs one trip to memory and there is little else to do, so 16
// (4 x 2 heads, 128 rows of 46 results: the call takes 21.0 us, with 4 at a time
// 25.4); once the rows fill the SMs, 4, whose fewer registers let more warps run (4096
// rows: 37.4 us, with 16 at a time 40.4).
template <int D, int kBatch>
__global__ void __launch_bounds__(256) attn_decode_merge_kernel(const DecodeParams p) {
  constexpr int kPer = D / 32;
  constexpr float kLog2e = 1.44269504088896340736f;
  const long long nrows = (long long)p.B * p.Hq * p.Lq;
  const long long row = (long long)blockIdx.x * (blockDim.x / 32) + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (row >= nrows) {  // warp-uniform
    wait_for_previous_kernel();
    return;
  }
  const int rows_all = p.group * p.Lq;
  const int bh = (int)(row / rows_all);
  const int r = (int)(row - (long long)bh * rows_all);
  const int b = bh / p.Hkv;
  const int units = p.Hkv * p.row_tiles;
  const int unit = (bh - b * p.Hkv) * p.row_tiles + r / p.tile_rows;
  const int rr = r % p.tile_rows;
  // the line's length, and what lies before sequence b
  int all = 0, before = 0;
#pragma unroll 4
  for (int i = lane; i < p.B; i += 32) {
    const int n = sched::cost_of(sched::seq_len(p.kv_lens, i, p.Lk), p.piece);
    all += n;
    if (i < b) before += n;
  }
  const int T = __reduce_add_sync(0xffffffffu, all) * units;
  before = __reduce_add_sync(0xffffffffu, before) * units;
  const int tiles = sched::tiles_of(sched::seq_len(p.kv_lens, b, p.Lk));
  // the unit's CTAs c0 .. c1, and how many partial results they left
  int c0 = 0, pieces = 0;
  if (tiles > 0) {
    const int first = before + unit * (tiles + p.piece) + p.piece;  // the unit's tile 0
    const sched::Split split(T, sched::ctas_used(T, p.num_ctas));
    c0 = split.of(first);
    pieces = split.of(first + tiles - 1) - c0 + 1;
  }
  // every thread waits, so that whatever follows this kernel follows the one before it
  wait_for_previous_kernel();
  if (p.num_prefix == 0 && pieces == 1) return;  // written by its CTA
  // result s of the row: the prefix's, then the unit's pieces (the start in slot 2 c0 + 1,
  // middles and end in 2 c) or, from one CTA, its row of own_o
  const int n = p.num_prefix + pieces;
  auto at = [&](int s, const float** o, const float** lse) {
    long long i;
    if (s < p.num_prefix) {
      i = s * nrows + row;
      *o = p.prefix_o;
      *lse = p.prefix_lse;
    } else if (pieces == 1) {
      i = row;
      *o = p.own_o;
      *lse = p.own_lse;
    } else {
      const int c = s - p.num_prefix;
      i = (long long)(2 * (c0 + c) + (c == 0 ? 1 : 0)) * p.tile_rows + rr;
      *o = p.ws_o;
      *lse = p.ws_lse;
    }
    *o += i * D + lane * kPer;
    *lse += i;
  };
  float v[kBatch][kPer];
  auto load = [&](int s0) {
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      if (s0 + u >= n) break;
      const float *po, *pl;
      at(s0 + u, &po, &pl);
      if constexpr (kPer == 4) {
        const float4 x = *reinterpret_cast<const float4*>(po);
        v[u][0] = x.x;
        v[u][1] = x.y;
        v[u][2] = x.z;
        v[u][3] = x.w;
      } else {
        const float2 x = *reinterpret_cast<const float2*>(po);
        v[u][0] = x.x;
        v[u][1] = x.y;
      }
    }
  };
  float acc[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) acc[i] = 0.0f;
  float mx = -INFINITY, sum = 0.0f;
  for (int s0 = 0; s0 < n; s0 += 32) {
    // lane i: LSE of result s0 + i
    float ls = -INFINITY;
    const float *po, *pl;
    if (s0 + lane < n) {
      at(s0 + lane, &po, &pl);
      ls = *pl;
    }
    load(s0);
    float m = ls;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    const bool none = m == -INFINITY && !__any_sync(0xffffffffu, ls != ls);  // NaN stays NaN
    if (none) continue;
    if (m > mx) {  // more than 32 results: what came before counts relative to the new maximum
      const float a = ptx::ex2((mx - m) * kLog2e);
      sum *= a;
#pragma unroll
      for (int i = 0; i < kPer; ++i) acc[i] *= a;
      mx = m;
    }
    const float wl = ptx::ex2((ls - mx) * kLog2e);  // 0 for -inf
    sum += wl;
    // a result without keys has no row (anything may lie there); one whose weight only
    // underflows has, and a NaN in it counts
    const uint32_t live = __ballot_sync(0xffffffffu, ls != -INFINITY);
    const int k = min(32, n - s0);
    for (int i0 = 0; i0 < k; i0 += kBatch) {
      if (i0 > 0) load(s0 + i0);
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        if (i0 + u >= k) break;
        const float wi = __shfl_sync(0xffffffffu, wl, i0 + u);
        const bool has = live >> (i0 + u) & 1u;
#pragma unroll
        for (int i = 0; i < kPer; ++i) acc[i] += has ? wi * v[u][i] : 0.0f;
      }
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  const float inv = sum != 0.0f ? 1.0f / sum : 0.0f;
  __nv_bfloat16* dst = reinterpret_cast<__nv_bfloat16*>(p.o) + row * D + lane * kPer;
  if constexpr (kPer == 4)
    *reinterpret_cast<uint2*>(dst) = make_uint2(ptx::pack_bf16x2(acc[0] * inv, acc[1] * inv),
                                                ptx::pack_bf16x2(acc[2] * inv, acc[3] * inv));
  else
    *reinterpret_cast<uint32_t*>(dst) = ptx::pack_bf16x2(acc[0] * inv, acc[1] * inv);
  if (lane == 0) p.lse[row] = sum != 0.0f ? mx + ptx::lg2(sum) * kLn2 : -INFINITY;
}

namespace {

// A kernel launch that may start before the kernel ahead of it in the stream has ended.
template <class... Args>
cudaError_t launch_early(void (*kern)(Args...), unsigned grid, unsigned threads, size_t smem,
                         cudaStream_t stream, bool early, const Args&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr = {};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = early ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kern, args...);
}

template <int D, int NB, bool kQ8>
cudaError_t launch_nb(const CUtensorMap& tk, const CUtensorMap& tv, const DecodeParams& p,
                      cudaStream_t stream) {
  using C = RowCfg<D, NB, kQ8>;
  auto kern = attn_decode_rows_kernel<D, NB, kQ8>;
  static PerContextOnce once;
  const cudaError_t e = once_per_context(once, [&](int) {
    return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmemAlloc);
  });
  if (e != cudaSuccess) return e;
  return launch_early(kern, (unsigned)p.num_ctas, C::kThreads, C::kSmemAlloc, stream,
                      p.num_prefix > 0, tk, tv, p);
}

}  // namespace

// Over an 8-bit cache (kQ8) or a bf16 one.  Behind the kernel of a shared prefix
// (num_prefix > 0) it may start before that one has ended: they do not touch each
// other's data.
template <int D, bool kQ8>
cudaError_t launch_decode_rows(const CUtensorMap& tk, const CUtensorMap& tv,
                               const DecodeParams& p, cudaStream_t stream) {
  if (p.tile_rows == 8) return launch_nb<D, 1, kQ8>(tk, tv, p, stream);
  if (p.tile_rows == 16) return launch_nb<D, 2, kQ8>(tk, tv, p, stream);
  if constexpr (D == 64)
    if (p.tile_rows == 32) return launch_nb<D, 4, kQ8>(tk, tv, p, stream);
  return cudaErrorInvalidValue;
}

// Launched so that its start overlaps the end of the decode kernel before it; it
// waits for that kernel's results itself.
template <int D>
cudaError_t launch_decode_merge(const DecodeParams& p, int num_sms, cudaStream_t stream) {
  const long long nrows = (long long)p.B * p.Hq * p.Lq;
  const unsigned grid = (unsigned)((nrows + 7) / 8);  // 8 rows per CTA
  if (grid <= 2u * (unsigned)num_sms)
    return launch_early(attn_decode_merge_kernel<D, 16>, grid, 256, 0, stream, true, p);
  return launch_early(attn_decode_merge_kernel<D, 4>, grid, 256, 0, stream, true, p);
}

template cudaError_t launch_decode_rows<64, true>(const CUtensorMap&, const CUtensorMap&,
                                                  const DecodeParams&, cudaStream_t);
template cudaError_t launch_decode_rows<128, true>(const CUtensorMap&, const CUtensorMap&,
                                                   const DecodeParams&, cudaStream_t);
template cudaError_t launch_decode_rows<64, false>(const CUtensorMap&, const CUtensorMap&,
                                                   const DecodeParams&, cudaStream_t);
template cudaError_t launch_decode_rows<128, false>(const CUtensorMap&, const CUtensorMap&,
                                                    const DecodeParams&, cudaStream_t);
template cudaError_t launch_decode_merge<64>(const DecodeParams&, int, cudaStream_t);
template cudaError_t launch_decode_merge<128>(const DecodeParams&, int, cudaStream_t);

// Rows of a TMA box: a warp's block, or a page shorter than it.
int decode_rows_box(int d, bool q8, int page_size) {
  return std::min(page_size, q8 || d == 64 ? 32 : 16);
}

}  // namespace attn
