// Split-KV decode over an 8-bit cache (format in cache_q8.cuh) for sm_100a.
//
//   S_ij = scale * 2^(ke_j - 127) * <q_i, kc_j>,   P = softmax(S),
//   O_i  = sum_j P_ij 2^(ve_j - 127) vc_j,         LSE_i = log sum_j exp(S_ij),
// kc_j, vc_j the e4m3 codes of key j.  The codes are never expanded in memory.
//
// What bounds it is the stream of codes (2 (d + 1) bytes per key and KV head for
// all query rows of the group), as long as turning codes into matrix operands is
// cheap.  Few query rows share a key (8 at Lq = 1 with 8 heads per group), so the
// work is laid out around that: a warp owns whole keys and computes the
// transposed products with mma.m16n8k16 (f16 in, fp32 out), whose N = 8 is the
// query rows and whose M = 16 is keys (S^T = K Q^T) or d (O^T = V^T P^T).  The
// codes go from shared memory to registers, two instructions turn four of them
// into two f16 pairs (exact), and these are the A operand: nothing is written
// back to shared memory, which the tcgen05 path would need (its operands live in
// shared or tensor memory, and expanding 1 byte to 2 there moves 5 bytes of
// shared-memory traffic per code).
//
// Numbers.  Q is scaled per row by a power of two into f16's upper range (an
// element keeps all 8 bits of its bf16 significand down to 2^-31 of the row's
// largest).  Scores, maxima and sums are fp32.  P times the value scale goes into
// the second product as f16 relative to a running reference of its own, R_i >=
// max_j (S_ij log2 e + ve_j) - 8, separate from the softmax's reference m_i: a
// value row with a large scale but a small weight then costs the others nothing.
// f16 rounds P to 11 bits, 8 times finer than bf16.
//
// Layout of a warp's unit of 32 keys (two blocks of 16).  A contraction does not
// care about the order of its terms, so d and the keys are permuted to let every
// thread read 16 (d = 64: 8, for V) consecutive bytes:
//   S^T: thread (g = lane / 4, t = lane % 4) reads d bytes 64 j + 16 t .. + 15 of
//     keys sigma(g) and 8 + sigma(g); word m of them is k-step 4 j + m.
//   O^T: it reads d bytes (d / 8) g .. of keys sigma(2t), sigma(2t + 1), + 8; a
//     byte permute of two keys' words pairs the keys, as the operand wants.
// sigma (a permutation of 0..7) makes both reads conflict-free in the swizzled
// tile; P^T comes from S^T by movmatrix (8x8 transposes), with no shared memory.
//
// Every warp streams its own 32-key blocks through its own ring (TMA boxes, one
// mbarrier per stage; lane 0 issues), so warps wait for one another only where a
// piece of work (q8_sched.cuh) ends and their results are merged; with 16-key pages
// as many lanes issue boxes as there are warps.  The ring runs on across pieces.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "attn_params.h"
#include "cache_q8.cuh"
#include "cache_q8_params.h"
#include "host_once.h"
#include "ptx.cuh"
#include "q8_sched.cuh"

namespace attn {
namespace {

constexpr int kUnit = 32;             // keys a warp takes at a time
constexpr float kSlack = 8.0f;        // log2 units a running reference may lag behind
constexpr float kLn2 = 0.69314718055994530942f;

// Warps per CTA (one CTA per SM): as many as the registers allow, since a warp's
// chain of dependent steps per block, not the issue rate, is what more warps hide.
template <int D, int NB>
struct Q8Cfg {
  static constexpr int kWarps = D == 128 ? (NB == 1 ? 12 : 8) : NB == 1 ? 16 : NB == 2 ? 12 : 8;
  static constexpr int kThreads = kWarps * 32;
  static constexpr int kRows = 8 * NB;          // query rows per unit
  static constexpr int kTileBytes = kUnit * D;  // one K or V block
  static constexpr int kStageBytes = 2 * kTileBytes;
  static constexpr int kStages = D == 128 ? 2 : NB == 4 ? 4 : 3;
  static constexpr int kRingBytes = kWarps * kStages * kStageBytes;
  // merge buffers: a warp's accumulators and statistics, one 128-byte row per register
  static constexpr int kMergeRegs = NB * (D / 16 * 4 + 6);
  static constexpr int kMergeBufs = kWarps == 12 ? 4 : kWarps / 2;
  static constexpr int kMergeBytes = kMergeBufs * kMergeRegs * 128;
  static constexpr int kOffMerge = kRingBytes;
  static constexpr int kOffExp = kOffMerge + kMergeBytes;  // [warp][stage][K, V][32] scale bytes
  static constexpr int kOffQ = kOffExp + kWarps * kStages * 64;  // Q of two pieces
  static constexpr int kOffBar = kOffQ + 2 * kRows * D * 2;
  static constexpr int kOffMisc = kOffBar + (kWarps * kStages + 2) * 8;
  static constexpr int kSmemBytes = kOffMisc + 64;
  static constexpr int kSmemAlloc = kSmemBytes + 1024;  // slack for 1024-byte alignment
  static_assert(kSmemAlloc <= 227 * 1024, "shared memory");
  };

// Key of mma row g inside its group of 8 (see the head of this file).
//   d = 128 (128-byte rows): sigma(2t + 1) = sigma(2t) ^ 4, and sigma(2t) >> 1 = t;
//   d = 64 (64-byte rows): sigma(2t + 1) = sigma(2t) ^ 3, sigma(2t) in {0, 1, 4, 5}.
template <int D>
__device__ __forceinline__ int sigma(int g) {
  if constexpr (D == 128) return ((g & 6) + (g >> 2)) ^ ((g & 1) << 2);
  return (((g >> 1) & 1) | (g & 4)) ^ (g & 1 ? 3 : 0);
}

// Byte offset of 16-byte chunk c of key row r in a unit as TMA lays it out
// (128-byte swizzle for 128-byte rows, 64-byte swizzle for 64-byte rows).
template <int D>
__device__ __forceinline__ uint32_t chunk_off(int r, int c) {
  if constexpr (D == 128) return (uint32_t)(r * 128 + ((c ^ (r & 7)) << 4));
  return (uint32_t)(r * 64 + ((c ^ ((r >> 1) & 3)) << 4));
}

__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
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

template <int D, int NB>
__global__ void __launch_bounds__(Q8Cfg<D, NB>::kThreads, 1)
    attn_decode_q8_kernel(const __grid_constant__ CUtensorMap tm_k,
                          const __grid_constant__ CUtensorMap tm_v, const DecodeQ8Params p) {
  using C = Q8Cfg<D, NB>;
  constexpr int S = C::kStages;
  constexpr int kWarps = C::kWarps;
  constexpr int kJ = D / 64;   // 16-byte K chunks per thread and key
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
  q8::Share* share = reinterpret_cast<q8::Share*>(smem + C::kOffMisc + 8);
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
    const q8::Share sh =
        q8::find_share(p.kv_lens, p.B, p.Lk, units, blockIdx.x, gridDim.x, p.err);
    if (lane == 0) {
      *share = sh;
      *abort_flag = 0;
    }
  } else if (threadIdx.x == 32) {
    ptx::prefetch_tmap(&tm_k);
    ptx::prefetch_tmap(&tm_v);
  }
  __syncthreads();
  q8::let_next_kernel_launch();

  // Q of a piece, one copy of its rows (they lie one after another) into buffer
  // piece % 2, by one thread a piece ahead.
  const int rows_all = p.group * p.Lq;
  int q_issued = 0;
  auto load_q = [&](const q8::Walk& a, int piece) {
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
  q8::Walk lw;
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
      if (j < l_end) {
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
    dst[lane] = (uint8_t)ke;
    dst[32 + lane] = (uint8_t)ve;
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
    if ((lane & (rows - 1)) == 0) {
      const int j = l_key + lane;
      const int y = paged ? j & (p.page_size - 1) : j;
      ptx::tma_load_3d_hint(kd + lane * D, &tm_k, &bars[s], 0, y, z, kv_policy);
      ptx::tma_load_3d_hint(vd + lane * D, &tm_v, &bars[s], 0, y, z, kv_policy);
    }
    ke = ve = 1;
    const int j = l_key + lane;
    if (j < l_end && z >= 0) {
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
      if (i < n_issued) store_exps(i, ke[i], ve[i]);
  }
  int pend_ke = 1, pend_ve = 1;  // scale bytes of the block issued last
  bool pending = false;          // not stored yet

  const int sg = sigma<D>(g), s2t0 = sigma<D>(2 * t), s2t1 = sigma<D>(2 * t + 1);
  bool ok = true;
  int done = 0;  // blocks consumed
  float* merge = reinterpret_cast<float*>(smem + C::kOffMerge);
  q8::Walk w;
  w.start(*share, p.kv_lens, p.Lk);
  if (threadIdx.x == 0 && w.valid()) load_q(w, 0);
  for (int piece = 0; w.valid(); ++piece) {
    q8::Walk next = w;  // the piece after this one
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
    uint32_t qf[NB][kJ * 4][2];
    float fac0[NB], fac1[NB];  // scale * log2 e * 2^(row shift) of query rows 2t and 2t + 1
    ok = ok && ptx::mbar_wait_a(ptx::smem_u32(&q_bars[piece & 1]), (uint32_t)(piece >> 1) & 1u,
                                abort_flag, p.err, kDevErrTimeoutProducer);
    const uint4* q_s =
        reinterpret_cast<const uint4*>(smem + C::kOffQ + (piece & 1) * (C::kRows * D * 2));
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      uint4 raw[kJ][2];
      const int r = nb * 8 + g;
#pragma unroll
      for (int j = 0; j < kJ; ++j)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          raw[j][h] =
              r < rows_valid ? q_s[r * (D / 8) + j * 8 + t * 2 + h] : make_uint4(0, 0, 0, 0);
      float amax = 0.0f;
#pragma unroll
      for (int j = 0; j < kJ; ++j)
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
      for (int j = 0; j < kJ; ++j)
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

    // ------------------------------------------------------------- key blocks
    float o[NB][kMu][4];
    float m[NB][2], R[NB][2], l[NB][2];
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
      for (int mu = 0; mu < kMu; ++mu)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[nb][mu][i] = 0.0f;
      m[nb][0] = m[nb][1] = R[nb][0] = R[nb][1] = -INFINITY;
      l[nb][0] = l[nb][1] = 0.0f;
    }
    for (int k0 = w.t0 * 128 + warp * kUnit; k0 < key_end && ok; k0 += kWarps * kUnit) {
      const int s = done % S;
      const int left = key_end - k0;  // visible keys of the block: [0, left)
      ok = ptx::mbar_wait_a(ptx::smem_u32(&bars[s]), (uint32_t)(done / S) & 1u, abort_flag, p.err,
                            kDevErrTimeoutProducer);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      if (pending) store_exps(n_issued - 1, pend_ke, pend_ve);
      __syncwarp();
      const uint32_t sk = ptx::smem_u32(ring + s * C::kStageBytes);
      const uint32_t sv = sk + C::kTileBytes;
      const uint8_t* eb = exps + s * 64;

      // S^T of both 16-key blocks
      float z[2][NB][4];
#pragma unroll
      for (int blk = 0; blk < 2; ++blk) {
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int i = 0; i < 4; ++i) z[blk][nb][i] = 0.0f;
#pragma unroll
        for (int j = 0; j < kJ; ++j) {
          uint32_t wa[4], wb[4];
          ptx::ld_shared_v4(sk + chunk_off<D>(blk * 16 + sg, j * 4 + t), wa[0], wa[1], wa[2], wa[3]);
          ptx::ld_shared_v4(sk + chunk_off<D>(blk * 16 + 8 + sg, j * 4 + t), wb[0], wb[1], wb[2],
                            wb[3]);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint32_t a0, a1, a2, a3;
            q8::codes4_to_f16(wa[i], a0, a2);
            q8::codes4_to_f16(wb[i], a1, a3);
#pragma unroll
            for (int nb = 0; nb < NB; ++nb)
              mma16816(z[blk][nb], a0, a1, a2, a3, qf[nb][j * 4 + i][0], qf[nb][j * 4 + i][1]);
          }
        }
      }
      // scores in the base-2 domain; z[..][i]: key blk * 16 + (i / 2) * 8 + sigma(g), row 2t + i % 2
      float vexp[2][2];
#pragma unroll
      for (int blk = 0; blk < 2; ++blk)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int key = blk * 16 + h * 8 + sg;
          const float ks = q8::scale_of(eb[key]);
          vexp[blk][h] = (float)((int)eb[32 + key] - 127);
          const bool vis = key < left;
#pragma unroll
          for (int nb = 0; nb < NB; ++nb) {
            z[blk][nb][2 * h] = vis ? z[blk][nb][2 * h] * (ks * fac0[nb]) : -INFINITY;
            z[blk][nb][2 * h + 1] = vis ? z[blk][nb][2 * h + 1] * (ks * fac1[nb]) : -INFINITY;
          }
        }
      // running references: raised only when a score passes one by more than kSlack
      bool need = false;
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float zm = fmaxf(fmaxf(z[0][nb][i], z[0][nb][2 + i]),
                                 fmaxf(z[1][nb][i], z[1][nb][2 + i]));
          const float wm = fmaxf(fmaxf(z[0][nb][i] + vexp[0][0], z[0][nb][2 + i] + vexp[0][1]),
                                 fmaxf(z[1][nb][i] + vexp[1][0], z[1][nb][2 + i] + vexp[1][1]));
          need |= zm > m[nb][i] + kSlack || wm > R[nb][i] + kSlack;
        }
      if (__any_sync(0xffffffffu, need)) {
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            float zm = fmaxf(fmaxf(z[0][nb][i], z[0][nb][2 + i]),
                             fmaxf(z[1][nb][i], z[1][nb][2 + i]));
            float wm = fmaxf(fmaxf(z[0][nb][i] + vexp[0][0], z[0][nb][2 + i] + vexp[0][1]),
                             fmaxf(z[1][nb][i] + vexp[1][0], z[1][nb][2 + i] + vexp[1][1]));
#pragma unroll
            for (int x = 4; x < 32; x <<= 1) {
              zm = fmaxf(zm, __shfl_xor_sync(0xffffffffu, zm, x));
              wm = fmaxf(wm, __shfl_xor_sync(0xffffffffu, wm, x));
            }
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
      uint32_t pb[2][NB][2];
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int blk = 0; blk < 2; ++blk)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const float z0 = z[blk][nb][2 * h], z1 = z[blk][nb][2 * h + 1];
            l[nb][0] += ptx::ex2(z0 - m[nb][0]);
            l[nb][1] += ptx::ex2(z1 - m[nb][1]);
            const float w0 = ptx::ex2(z0 + vexp[blk][h] - R[nb][0]);
            const float w1 = ptx::ex2(z1 + vexp[blk][h] - R[nb][1]);
            pb[blk][nb][h] = transpose8x8(pack_f16x2(w0, w1));
          }
      // O^T += V^T P^T
#pragma unroll
      for (int blk = 0; blk < 2; ++blk) {
        const int ka = blk * 16 + s2t0, kb = blk * 16 + s2t1;
        constexpr int kW = D / 32;  // words per thread and key
        uint32_t vw[4][kW];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int key = (i & 1 ? kb : ka) + (i >> 1) * 8;
          if constexpr (D == 128)
            ptx::ld_shared_v4(sv + chunk_off<D>(key, g), vw[i][0], vw[i][1], vw[i][2], vw[i][3]);
          else
            ld_shared_v2(sv + chunk_off<D>(key, g >> 1) + (g & 1) * 8, vw[i][0], vw[i][1]);
          // a masked key's codes may be anything (even NaN): 0 * NaN would poison O
          if (left < kUnit && key >= left) {
#pragma unroll
            for (int x = 0; x < kW; ++x) vw[i][x] = 0u;
          }
        }
#pragma unroll
        for (int x = 0; x < kW; ++x)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint32_t sel = h ? 0x7362 : 0x5140;  // bytes 2h, 2h + 1 of both keys, interleaved
            uint32_t a0, a1, a2, a3;
            q8::codes4_to_f16(__byte_perm(vw[0][x], vw[1][x], sel), a0, a1);
            q8::codes4_to_f16(__byte_perm(vw[2][x], vw[3][x], sel), a2, a3);
#pragma unroll
            for (int nb = 0; nb < NB; ++nb)
              mma16816(o[nb][2 * x + h], a0, a1, a2, a3, pb[blk][nb][0], pb[blk][nb][1]);
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
            const float mu0 = mn == -INFINITY ? 0.0f : mn, Ru0 = Rn == -INFINITY ? 0.0f : Rn;
            l[nb][i] = l[nb][i] * ptx::ex2(m[nb][i] - mu0) +
                       src[(nb * 6 + 4 + i) * 32] * ptx::ex2(m1 - mu0);
            a0[i] = ptx::ex2(R[nb][i] - Ru0);
            a1[i] = ptx::ex2(R1 - Ru0);
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
      float M = -INFINITY, Rm = -INFINITY;
#pragma unroll
      for (int x = 0; x < C::kMergeBufs; ++x)
        if (x < n) {
          M = fmaxf(M, st[x * C::kMergeRegs * 32]);
          Rm = fmaxf(Rm, st[x * C::kMergeRegs * 32 + 64]);
        }
      const float Mu = M == -INFINITY ? 0.0f : M, Ru = Rm == -INFINITY ? 0.0f : Rm;
      float ls = 0.0f, v0 = 0.0f, v1 = 0.0f;
#pragma unroll
      for (int x = 0; x < C::kMergeBufs; ++x)
        if (x < n) {
          const int off = x * C::kMergeRegs * 32;
          ls += st[off + 128] * ptx::ex2(st[off] - Mu);
          const float a = ptx::ex2(st[off + 64] - Ru);
          v0 += a * ov[off];
          v1 += a * ov[off + 64];
        }
#pragma unroll
      for (int x = 4; x < 32; x <<= 1) ls += __shfl_xor_sync(0xffffffffu, ls, x);
      const bool have = ok && ls > 0.0f;
      const float inv = have ? 1.0f / ls : 0.0f;
      const float f = ptx::ex2(Ru - Mu);  // O is in units of 2^R, l in units of 2^m
      v0 = v0 * inv * f;
      v1 = v1 * inv * f;
      const int r = nb * 8 + 2 * t + i;
      if (r < rows_valid) {
        const long long to = (at + r) * D + g * (D / 8) + 2 * mu;
        if (final)
          *reinterpret_cast<uint32_t*>(reinterpret_cast<__nv_bfloat16*>(p.o) + to) =
              ptx::pack_bf16x2(v0, v1);
        else
          *reinterpret_cast<float2*>(p.ws_o + to) = make_float2(v0, v1);
        if (mu == 0 && g == 0)
          (final ? p.lse : p.ws_lse)[at + r] = have ? (Mu + ptx::lg2(ls)) * kLn2 : -INFINITY;
      }
    }
    if (!ok) break;
    w = next;
  }
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

// Returns once the kernel before this one in the stream is complete and its writes
// are visible (this one may have started earlier).
__device__ __forceinline__ void wait_for_previous_kernel() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

// Merges the pieces of units that several CTAs computed,
//   LSE = log sum_s exp(LSE_s),  O = sum_s exp(LSE_s - LSE) O_s,
// and writes the empty result of sequences without keys.  One warp per output row;
// lane i owns d / 32 consecutive elements.
template <int D>
__global__ void __launch_bounds__(256) attn_decode_q8_combine_kernel(const DecodeQ8Params p) {
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
  for (int i = lane; i < p.B; i += 32) {
    const int n = q8::cost_of(q8::seq_len(p.kv_lens, i, p.Lk));
    all += n;
    if (i < b) before += n;
  }
  const int T = __reduce_add_sync(0xffffffffu, all) * units;
  before = __reduce_add_sync(0xffffffffu, before) * units;
  const int tiles = q8::tiles_of(q8::seq_len(p.kv_lens, b, p.Lk));
  // every thread waits, so that whatever follows this kernel follows the one before it
  wait_for_previous_kernel();
  __nv_bfloat16* dst = reinterpret_cast<__nv_bfloat16*>(p.o) + row * D + lane * kPer;
  float acc[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) acc[i] = 0.0f;
  float lse = -INFINITY;
  if (tiles > 0) {
    const int first = before + unit * (tiles + kQ8Piece) + kQ8Piece;  // the unit's tile 0
    const q8::Split split(T, q8::ctas_used(T, p.num_ctas));
    const int c0 = split.of(first), c1 = split.of(first + tiles - 1);
    if (c0 == c1) return;  // written by its CTA
    const int n = c1 - c0 + 1;
    // piece i of the unit: the start (slot 2 c0 + 1), then the ends and middles (2 c)
    auto slot_row = [&](int i) {
      return (long long)(2 * (c0 + i) + (i == 0 ? 1 : 0)) * p.tile_rows + rr;
    };
    float mx = -INFINITY;
    for (int i = lane; i < n; i += 32) mx = fmaxf(mx, p.ws_lse[slot_row(i)]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    float sum = 0.0f;
    if (mx != -INFINITY) {
      for (int i0 = 0; i0 < n; i0 += 32) {
        const float ls = i0 + lane < n ? p.ws_lse[slot_row(i0 + lane)] : -INFINITY;
        const float wl = ls == -INFINITY ? 0.0f : ptx::ex2((ls - mx) * kLog2e);
        sum += wl;
        const int k = min(32, n - i0);
#pragma unroll 4
        for (int i = 0; i < k; ++i) {
          const float wi = __shfl_sync(0xffffffffu, wl, i);
          const float* src = p.ws_o + slot_row(i0 + i) * D + lane * kPer;
          if constexpr (kPer == 4) {
            const float4 v = *reinterpret_cast<const float4*>(src);
            acc[0] += wi * v.x;
            acc[1] += wi * v.y;
            acc[2] += wi * v.z;
            acc[3] += wi * v.w;
          } else {
            const float2 v = *reinterpret_cast<const float2*>(src);
            acc[0] += wi * v.x;
            acc[1] += wi * v.y;
          }
        }
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      const float inv = 1.0f / sum;  // the piece of LSE mx has weight 1
#pragma unroll
      for (int i = 0; i < kPer; ++i) acc[i] *= inv;
      lse = mx + ptx::lg2(sum) * kLn2;
    }
  }
  if constexpr (kPer == 4)
    *reinterpret_cast<uint2*>(dst) =
        make_uint2(ptx::pack_bf16x2(acc[0], acc[1]), ptx::pack_bf16x2(acc[2], acc[3]));
  else
    *reinterpret_cast<uint32_t*>(dst) = ptx::pack_bf16x2(acc[0], acc[1]);
  if (lane == 0) p.lse[row] = lse;
}

namespace {

template <int D, int NB>
cudaError_t launch_nb(const CUtensorMap& tk, const CUtensorMap& tv, const DecodeQ8Params& p,
                      cudaStream_t stream) {
  using C = Q8Cfg<D, NB>;
  auto kern = attn_decode_q8_kernel<D, NB>;
  static PerContextOnce once;
  const cudaError_t e = once_per_context(once, [&](int) {
    return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmemAlloc);
  });
  if (e != cudaSuccess) return e;
  kern<<<p.num_ctas, C::kThreads, C::kSmemAlloc, stream>>>(tk, tv, p);
  return cudaGetLastError();
}

}  // namespace

template <int D>
cudaError_t launch_decode_q8(const CUtensorMap& tk, const CUtensorMap& tv,
                             const DecodeQ8Params& p, cudaStream_t stream) {
  if (p.tile_rows == 8) return launch_nb<D, 1>(tk, tv, p, stream);
  if (p.tile_rows == 16) return launch_nb<D, 2>(tk, tv, p, stream);
  if constexpr (D == 64)
    if (p.tile_rows == 32) return launch_nb<D, 4>(tk, tv, p, stream);
  return cudaErrorInvalidValue;
}

// Launched so that its start overlaps the end of the decode kernel before it; it
// waits for that kernel's results itself.
template <int D>
cudaError_t launch_decode_q8_combine(const DecodeQ8Params& p, cudaStream_t stream) {
  const long long nrows = (long long)p.B * p.Hq * p.Lq;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((nrows + 7) / 8));
  cfg.blockDim = dim3(256);
  cfg.stream = stream;
  cudaLaunchAttribute attr = {};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, attn_decode_q8_combine_kernel<D>, p);
}

template cudaError_t launch_decode_q8<64>(const CUtensorMap&, const CUtensorMap&,
                                          const DecodeQ8Params&, cudaStream_t);
template cudaError_t launch_decode_q8<128>(const CUtensorMap&, const CUtensorMap&,
                                           const DecodeQ8Params&, cudaStream_t);
template cudaError_t launch_decode_q8_combine<64>(const DecodeQ8Params&, cudaStream_t);
template cudaError_t launch_decode_q8_combine<128>(const DecodeQ8Params&, cudaStream_t);

// Rows of a TMA box over the codes: a warp's block, or a page shorter than it.
int decode_q8_box_rows(int page_size) { return page_size < kUnit ? page_size : kUnit; }

}  // namespace attn
