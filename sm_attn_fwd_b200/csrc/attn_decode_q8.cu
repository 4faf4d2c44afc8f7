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
// Every warp streams its own units through its own ring (TMA boxes, one mbarrier
// per stage; lane 0 issues), so warps never wait for one another until the merge
// at the end of the CTA: with 16-key pages eight lanes issue the boxes at once.
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

namespace attn {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kUnit = 32;             // keys a warp takes at a time
constexpr float kSlack = 8.0f;        // log2 units a running reference may lag behind
constexpr float kLn2 = 0.69314718055994530942f;

template <int D, int NB>
struct Q8Cfg {
  static constexpr int kRows = 8 * NB;            // query rows per CTA
  static constexpr int kTileBytes = kUnit * D;    // one K or V unit
  static constexpr int kStageBytes = 2 * kTileBytes;
  static constexpr int kStages = D == 128 ? 3 : 6;
  static constexpr int kRingBytes = kWarps * kStages * kStageBytes;
  static constexpr int kMergeBytes = kWarps * kRows * (D + 4) * 4 + kWarps * kRows * 12;
  static constexpr int kDataBytes = kRingBytes > kMergeBytes ? kRingBytes : kMergeBytes;
  static constexpr int kOffBar = kDataBytes;
  static constexpr int kOffAbort = kOffBar + kWarps * kStages * 8;
  static constexpr int kSmemBytes = kOffAbort + 16;
  static constexpr int kSmemAlloc = kSmemBytes + 1024;  // slack for 1024-byte alignment
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

__device__ __forceinline__ void ld_shared_v2(uint32_t addr, uint32_t& a, uint32_t& b) {
  asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(a), "=r"(b) : "r"(addr));
}

}  // namespace

template <int D, int NB>
__global__ void __launch_bounds__(kThreads, 1)
    attn_decode_q8_kernel(const __grid_constant__ CUtensorMap tm_k,
                          const __grid_constant__ CUtensorMap tm_v, const DecodeQ8Params p) {
  using C = Q8Cfg<D, NB>;
  constexpr int S = C::kStages;
  constexpr int kJ = D / 64;   // 16-byte K chunks per thread and key
  constexpr int kMu = D / 16;  // M tiles of O^T
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;

  // ------------------------------------------------------------ work unit
  // blockIdx.x = ((b * Hkv + hkv) * nsplit + split) * row_tiles + rt: the row
  // tiles that read the same keys are neighbours and share them through L2
  int idx = blockIdx.x;
  const int rt = idx % p.row_tiles;
  idx /= p.row_tiles;
  const int split = idx % p.nsplit;
  const int bh = idx / p.nsplit;
  const int b = bh / p.Hkv;
  const int hkv = bh - b * p.Hkv;
  int kv_len = p.kv_lens[b];
  if (kv_len < 0 || kv_len > p.Lk) {
    if (threadIdx.x == 0 && split == 0 && rt == 0) atomicOr(p.err, kDevErrBadKvLen);
    kv_len = kv_len < 0 ? 0 : p.Lk;
  }
  const int c0 = split * p.chunk;
  const int key_end = min(c0 + p.chunk, kv_len);
  const int rows_all = p.group * p.Lq;
  const int rows_valid = min(C::kRows, rows_all - rt * C::kRows);
  const long long row0 = (long long)bh * rows_all + (long long)rt * C::kRows;  // flat output row
  const long long nrows = (long long)p.B * p.Hq * p.Lq;
  if (c0 >= kv_len) {
    // no key of the sequence: weight 0 for the combine, or the empty result
    if ((int)threadIdx.x < rows_valid) {
      if (p.nsplit > 1)
        p.ws_lse[(long long)split * nrows + row0 + threadIdx.x] = -INFINITY;
      else
        p.lse[row0 + threadIdx.x] = -INFINITY;
    }
    if (p.nsplit == 1) {
      uint4* dst = reinterpret_cast<uint4*>(p.o) + row0 * (D / 8);
      for (int i = threadIdx.x; i < rows_valid * (D / 8); i += kThreads)
        dst[i] = make_uint4(0, 0, 0, 0);
    }
    return;  // uniform exit
  }

  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::kOffBar) + warp * S;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::kOffAbort);
  if (lane == 0) {
    for (int s = 0; s < S; ++s) ptx::mbar_init(&bars[s], 1);
    ptx::fence_mbar_init();
  }
  if (threadIdx.x == 0) {
    *abort_flag = 0;
    ptx::prefetch_tmap(&tm_k);
    ptx::prefetch_tmap(&tm_v);
  }
  __syncthreads();

  // ------------------------------------------------------------------ loads
  const int n_units_all = (key_end - c0 + kUnit - 1) / kUnit;
  const int n_mine = n_units_all > warp ? (n_units_all - warp + kWarps - 1) / kWarps : 0;
  uint8_t* ring = smem + warp * S * C::kStageBytes;
  const bool paged = p.block_table != nullptr;
  const int32_t* table = paged ? p.block_table + (long long)b * p.pages_per_seq : nullptr;
  const uint64_t kv_policy = ptx::l2_policy_evict_first();
  // first key of this warp's unit i
  auto unit_key = [&](int i) { return c0 + (warp + i * kWarps) * kUnit; };
  // pool index (page * Hkv + hkv) of the page that holds key j, or -1 (reads as zeros)
  auto pool = [&](int j) -> int {
    const int pi = j >> p.page_shift;
    if (pi >= p.pages_per_seq) return -1;
    const int page = __ldg(table + pi);
    if (page < 0 || page >= p.num_pages) {
      atomicOr(p.err, kDevErrBadPage);
      return -1;
    }
    return page * p.Hkv + hkv;
  };
  // Lane 0 issues unit i's boxes: one per operand, or one per page slice for
  // pages shorter than a unit.
  auto issue = [&](int i) {
    const int s = i % S;
    const uint32_t bar = ptx::smem_u32(&bars[s]);
    uint8_t* kd = ring + s * C::kStageBytes;
    uint8_t* vd = kd + C::kTileBytes;
    const int k0 = unit_key(i);
    ptx::mbar_arrive_expect_tx_a(bar, C::kStageBytes);
    if (!paged) {
      ptx::tma_load_3d_hint(kd, &tm_k, &bars[s], 0, k0, bh, kv_policy);
      ptx::tma_load_3d_hint(vd, &tm_v, &bars[s], 0, k0, bh, kv_policy);
    } else if (p.page_size >= kUnit) {
      const int z = pool(k0), y = k0 & (p.page_size - 1);
      ptx::tma_load_3d_hint(kd, &tm_k, &bars[s], 0, y, z, kv_policy);
      ptx::tma_load_3d_hint(vd, &tm_v, &bars[s], 0, y, z, kv_policy);
    } else {
      for (int r = 0; r < kUnit; r += p.page_size) {
        const int z = k0 + r < key_end ? pool(k0 + r) : -1;  // ids past the last page: never read
        ptx::tma_load_3d_hint(kd + r * D, &tm_k, &bars[s], 0, 0, z, kv_policy);
        ptx::tma_load_3d_hint(vd + r * D, &tm_v, &bars[s], 0, 0, z, kv_policy);
      }
    }
  };
  // Lane l's scale bytes of unit i's key l (keys past the end: any valid byte)
  auto load_exps = [&](int i, int& ke, int& ve) {
    ke = ve = 127;
    const int j = unit_key(i) + lane;
    if (i >= n_mine || j >= key_end) return;
    long long at;
    if (!paged) {
      at = (long long)bh * p.Lk + j;
    } else {
      const int z = pool(j);
      if (z < 0) return;
      at = ((long long)z << p.page_shift) + (j & (p.page_size - 1));
    }
    ke = __ldg(p.k_exp + at);
    ve = __ldg(p.v_exp + at);
  };
  int n_issued = min(n_mine, S);
  if (lane == 0)
    for (int i = 0; i < n_issued; ++i) issue(i);
  int ke_next, ve_next;
  load_exps(0, ke_next, ve_next);

  // ------------------------------------------------------------------- Q
  // B operand of S^T: query row n = g of each 8-row block, d in the order above
  uint32_t qf[NB][kJ * 4][2];
  float fac0[NB], fac1[NB];  // scale * log2 e * 2^(row shift) of query rows 2t and 2t + 1
#pragma unroll
  for (int nb = 0; nb < NB; ++nb) {
    uint4 raw[kJ][2];
    const int r = nb * 8 + g;
#pragma unroll
    for (int j = 0; j < kJ; ++j)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        raw[j][h] = r < rows_valid
                        ? __ldg(reinterpret_cast<const uint4*>(p.q) + (row0 + r) * (D / 8) +
                                j * 8 + t * 2 + h)
                        : make_uint4(0, 0, 0, 0);
    float amax = 0.0f;
#pragma unroll
    for (int j = 0; j < kJ; ++j)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t w[4] = {raw[j][h].x, raw[j][h].y, raw[j][h].z, raw[j][h].w};
#pragma unroll
        for (int i = 0; i < 4; ++i)
          amax = fmaxf(amax, fmaxf(fabsf(__uint_as_float(w[i] << 16)),
                                   fabsf(__uint_as_float(w[i] & 0xffff0000u))));
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
        const uint32_t w[4] = {raw[j][h].x, raw[j][h].y, raw[j][h].z, raw[j][h].w};
#pragma unroll
        for (int i = 0; i < 4; ++i)
          qf[nb][j * 4 + h * 2 + (i >> 1)][i & 1] =
              pack_f16x2(__uint_as_float(w[i] << 16) * s1 * s2,
                         __uint_as_float(w[i] & 0xffff0000u) * s1 * s2);
      }
    // rows 2t and 2t + 1 live in lanes 8t and 8t + 4
    const int sh0 = __shfl_sync(0xffffffffu, sh, 8 * t);
    const int sh1 = __shfl_sync(0xffffffffu, sh, 8 * t + 4);
    fac0[nb] = p.scale_log2 * __uint_as_float((uint32_t)(127 - sh0 / 2) << 23) *
               __uint_as_float((uint32_t)(127 - (sh0 - sh0 / 2)) << 23);
    fac1[nb] = p.scale_log2 * __uint_as_float((uint32_t)(127 - sh1 / 2) << 23) *
               __uint_as_float((uint32_t)(127 - (sh1 - sh1 / 2)) << 23);
  }

  // --------------------------------------------------------------- main loop
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
  const int sg = sigma<D>(g), s2t0 = sigma<D>(2 * t), s2t1 = sigma<D>(2 * t + 1);
  bool ok = true;
  int done = 0;
  for (; done < n_mine; ++done) {
    const int s = done % S;
    const int k0 = unit_key(done);
    const int left = key_end - k0;  // visible keys of the unit: [0, left)
    const int ke = ke_next, ve = ve_next;
    load_exps(done + 1, ke_next, ve_next);
    ok = ptx::mbar_wait_a(ptx::smem_u32(&bars[s]), (uint32_t)(done / S) & 1u, abort_flag, p.err,
                          kDevErrTimeoutProducer);
    ok = __all_sync(0xffffffffu, ok);
    if (!ok) break;
    const uint32_t sk = ptx::smem_u32(ring + s * C::kStageBytes);
    const uint32_t sv = sk + C::kTileBytes;

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
        const float ks = q8::scale_of(__shfl_sync(0xffffffffu, ke, key));
        vexp[blk][h] = (float)(__shfl_sync(0xffffffffu, ve, key) - 127);
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
      uint32_t w[4][kW];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int key = (i & 1 ? kb : ka) + (i >> 1) * 8;
        if constexpr (D == 128)
          ptx::ld_shared_v4(sv + chunk_off<D>(key, g), w[i][0], w[i][1], w[i][2], w[i][3]);
        else
          ld_shared_v2(sv + chunk_off<D>(key, g >> 1) + (g & 1) * 8, w[i][0], w[i][1]);
        // a masked key's codes may be anything (even NaN): 0 * NaN would poison O
        if (left < kUnit && key >= left) {
#pragma unroll
          for (int x = 0; x < kW; ++x) w[i][x] = 0u;
        }
      }
#pragma unroll
      for (int x = 0; x < kW; ++x)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t sel = h ? 0x7362 : 0x5140;  // bytes 2h, 2h + 1 of both keys, interleaved
          uint32_t a0, a1, a2, a3;
          q8::codes4_to_f16(__byte_perm(w[0][x], w[1][x], sel), a0, a1);
          q8::codes4_to_f16(__byte_perm(w[2][x], w[3][x], sel), a2, a3);
#pragma unroll
          for (int nb = 0; nb < NB; ++nb)
            mma16816(o[nb][2 * x + h], a0, a1, a2, a3, pb[blk][nb][0], pb[blk][nb][1]);
        }
    }
    // every lane has read the stage: the next unit may land there
    __syncwarp();
    if (done + S < n_mine) {
      if (lane == 0) issue(done + S);
      ++n_issued;
    }
  }
  if (!ok && lane == 0) {
    // a wait gave up: let the copies in flight land before the CTA goes on
    for (int i = done; i < n_issued; ++i) {
      int dummy = 0;
      ptx::mbar_wait_a(ptx::smem_u32(&bars[i % S]), (uint32_t)(i / S) & 1u, &dummy, nullptr, 0);
    }
  }

  // ------------------------------------------------------------------ merge
  // Each warp leaves O (in units of 2^R), m, R and l of its rows in shared
  // memory (the ring's); rows are padded by 4 floats against bank conflicts.
  constexpr int kLd = D + 4;
  float* mo = reinterpret_cast<float*>(smem);
  float* stat = mo + kWarps * C::kRows * kLd;  // [3][warp][row]
  __syncthreads();
#pragma unroll
  for (int nb = 0; nb < NB; ++nb)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float ls = l[nb][i];
#pragma unroll
      for (int x = 4; x < 32; x <<= 1) ls += __shfl_xor_sync(0xffffffffu, ls, x);
      const int r = nb * 8 + 2 * t + i;
      if (g == 0) {
        stat[warp * C::kRows + r] = m[nb][i];
        stat[(kWarps + warp) * C::kRows + r] = R[nb][i];
        stat[(2 * kWarps + warp) * C::kRows + r] = ls;
      }
      // d of o[nb][mu][i] and o[nb][mu][2 + i]: (D / 8) g + 2 mu, + 1
      float* dst = mo + (warp * C::kRows + r) * kLd + g * (D / 8);
#pragma unroll
      for (int mu = 0; mu < kMu; mu += 2)
        *reinterpret_cast<float4*>(dst + 2 * mu) =
            make_float4(o[nb][mu][i], o[nb][mu][2 + i], o[nb][mu + 1][i], o[nb][mu + 1][2 + i]);
    }
  __syncthreads();
  for (int i = threadIdx.x; i < rows_valid * (D / 4); i += kThreads) {
    const int r = i / (D / 4), c = i - r * (D / 4);
    float M = -INFINITY, Rm = -INFINITY;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      M = fmaxf(M, stat[w * C::kRows + r]);
      Rm = fmaxf(Rm, stat[(kWarps + w) * C::kRows + r]);
    }
    const float Mu = M == -INFINITY ? 0.0f : M, Ru = Rm == -INFINITY ? 0.0f : Rm;
    float L = 0.0f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      L += stat[(2 * kWarps + w) * C::kRows + r] * ptx::ex2(stat[w * C::kRows + r] - Mu);
      const float a = ptx::ex2(stat[(kWarps + w) * C::kRows + r] - Ru);
      const float4 v = *reinterpret_cast<const float4*>(mo + (w * C::kRows + r) * kLd + c * 4);
      acc.x += a * v.x;
      acc.y += a * v.y;
      acc.z += a * v.z;
      acc.w += a * v.w;
    }
    const float inv = L > 0.0f ? 1.0f / L : 0.0f;
    const float f = ptx::ex2(Ru - Mu);  // O is in units of 2^R, L in units of 2^m
    acc.x = acc.x * inv * f;
    acc.y = acc.y * inv * f;
    acc.z = acc.z * inv * f;
    acc.w = acc.w * inv * f;
    const long long row = row0 + r;
    if (p.nsplit > 1) {
      *reinterpret_cast<float4*>(p.ws_o + ((long long)split * nrows + row) * D + c * 4) = acc;
    } else {
      uint2 v;
      v.x = ptx::pack_bf16x2(acc.x, acc.y);
      v.y = ptx::pack_bf16x2(acc.z, acc.w);
      *reinterpret_cast<uint2*>(reinterpret_cast<__nv_bfloat16*>(p.o) + row * D + c * 4) = v;
    }
    if (c == 0) {
      const float lse = L > 0.0f ? (Mu + ptx::lg2(L)) * kLn2 : -INFINITY;
      if (p.nsplit > 1)
        p.ws_lse[(long long)split * nrows + row] = lse;
      else
        p.lse[row] = lse;
    }
  }
}

namespace {

template <int D, int NB>
cudaError_t launch_nb(const CUtensorMap& tk, const CUtensorMap& tv, DecodeQ8Params p,
                      cudaStream_t stream) {
  auto kern = attn_decode_q8_kernel<D, NB>;
  constexpr int smem = Q8Cfg<D, NB>::kSmemAlloc;
  static PerContextOnce once;
  const cudaError_t e = once_per_context(once, [&](int) {
    return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  });
  if (e != cudaSuccess) return e;
  const int rows = p.group * p.Lq;
  p.row_tiles = (rows + 8 * NB - 1) / (8 * NB);
  const long long grid = (long long)p.B * p.Hkv * p.nsplit * p.row_tiles;
  if (grid > 0x7fffffffLL) return cudaErrorInvalidValue;
  kern<<<(unsigned)grid, kThreads, smem, stream>>>(tk, tv, p);
  return cudaGetLastError();
}

}  // namespace

// Query rows per CTA: 8, 16 or 32, the smallest that holds the group's rows (32
// is the most whose accumulators fit in the registers); more rows take several
// row tiles, which read the same keys through L2.
template <int D>
cudaError_t launch_decode_q8(const CUtensorMap& tk, const CUtensorMap& tv,
                             const DecodeQ8Params& p, cudaStream_t stream) {
  const long long rows = (long long)p.group * p.Lq;
  if (rows <= 8) return launch_nb<D, 1>(tk, tv, p, stream);
  if (rows <= 16) return launch_nb<D, 2>(tk, tv, p, stream);
  return launch_nb<D, 4>(tk, tv, p, stream);
}

template cudaError_t launch_decode_q8<64>(const CUtensorMap&, const CUtensorMap&,
                                          const DecodeQ8Params&, cudaStream_t);
template cudaError_t launch_decode_q8<128>(const CUtensorMap&, const CUtensorMap&,
                                           const DecodeQ8Params&, cudaStream_t);

// Rows of a TMA box over the codes: a warp's unit, or a page shorter than it.
int decode_q8_box_rows(int page_size) { return page_size < kUnit ? page_size : kUnit; }

}  // namespace attn
