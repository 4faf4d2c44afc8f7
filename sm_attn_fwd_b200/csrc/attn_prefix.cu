// Decode over a prefix that every sequence of the batch shares, for sm_100a.
//
// All B * Hq / Hkv * Lq query rows of a KV head attend to the same keys, so they
// are stacked into 128-row tiles whatever sequence they belong to, and each key
// tile is read once for all of them: O_s = softmax(Q K_s^T * scale) V_s and its
// log-sum-exp per split s of the prefix, left as a partial result beside those of
// the sequences' own caches for the combine kernel (attn_kernels.cu).  Reading the
// prefix per sequence instead would move B times its bytes.
//
// Work: 4 d flops per (row, key) on 4 d bytes per key and KV head, so with R rows
// per KV head the intensity is R flops per byte: past about 250 rows the tensor
// cores (and, as in the prefill, the exponentials of the softmax) bound it, below
// that HBM does.  Measured: 32768 keys of d = 128, 8 KV heads, 512 rows each: 81 us, 850
// TFLOP/s or 51 % of the measured peak (tensor pipe 47 %, exponentials 47 %, a softmax
// warpgroup's chain from S to P in between, as in the prefill); DRAM reads 135 MB, the
// prefix once.
//
// A CTA takes one (KV head, split, pair of row tiles) and runs the prefill's
// pipeline on it without its masks and schedules: warp 0 loads (Q_A, Q_B and a ring
// of K/V tiles), warp 1 issues the MMAs of tile A and warp 2 those of tile B, and
// two warpgroups turn S into P, taking turns on the exponentials; one K/V stream
// feeds both tiles.  CTAs that differ in the row pair only are neighbours in the
// grid, so the other pairs' reads of the same keys hit L2.  Tensor memory: S_A
// [0,128), S_B [128,256), O_A at 256, O_B at 256 + d; P over S for d = 128, in
// columns of its own for d = 64.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "attn_params.h"
#include "attn_prefix_params.h"
#include "decode_sched.cuh"
#include "host_once.h"
#include "ptx.cuh"
#include "softmax_row.cuh"

namespace attn {
namespace {

constexpr int kThreads = 384;
constexpr int kRegsLow = 80;    // warpgroup 0; 80*128 + 2*208*128 <= 168*384
constexpr int kRegsHigh = 208;  // softmax warpgroups
constexpr int kTmemCols = 512;
constexpr float kRescaleThreshold = 8.0f;  // log2 units: rescale O when the max grows by > 2^8
constexpr float kLn2 = 0.69314718055994530942f;

template <int D>
struct Cfg {
  static constexpr int kAtoms = D / 64;
  static constexpr int kAtomBytes = 128 * 128;
  static constexpr int kTileBytes = 128 * D * 2;
  static constexpr int kStages = (D == 64) ? 4 : 2;
  static constexpr bool kSepP = (D == 64);  // P has tensor-memory columns of its own
  static constexpr int kOffQ = 0;           // Q_A, Q_B
  static constexpr int kOffK = 2 * kTileBytes;
  static constexpr int kOffV = kOffK + kStages * kTileBytes;
  static constexpr int kOffBar = kOffV + kStages * kTileBytes;
  static constexpr int kNumBars = 13 + 4 * kStages;
  static constexpr int kOffMisc = kOffBar + ((kNumBars * 8 + 15) / 16) * 16;
  static constexpr int kSmemBytes = kOffMisc + 64;
  static constexpr int kSmemAlloc = kSmemBytes + 1024;
};

struct Misc {
  uint32_t tmem_base;
  int abort;
};

// Barrier slots; [2] = one per query tile.
enum : int {
  kQFull = 0,   // [2] TMA -> MMA: Q_x landed
  kSFull = 2,   // [2] MMA -> softmax x: S_x ready
  kSFree = 4,   // [2] softmax x (128) -> MMA: S_x loaded into registers (separate P)
  kPFull = 6,   // [2] softmax x (128) -> MMA: P_x written, O_x rescaled
  kODone = 8,   // [2] MMA -> softmax x: P_x V done
  kTurn = 10,   // [2] softmax 1-x (128) -> softmax x: x may run its exponentials
  kDrain = 12,  // MMA warps: all MMAs done
  kKv = 13,     // k_full[S], k_empty[S], v_full[S], v_empty[S]
};

__device__ __forceinline__ void tma_load_4d_a(uint32_t dst, const void* tmap, uint32_t bar, int x,
                                              int y, int z, int w) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(tmap)), "r"(bar), "r"(x), "r"(y), "r"(z), "r"(w)
      : "memory");
}

}  // namespace

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    attn_prefix_kernel(const __grid_constant__ CUtensorMap tm_q,
                       const __grid_constant__ CUtensorMap tm_k,
                       const __grid_constant__ CUtensorMap tm_v, const PrefixParams p) {
  using C = Cfg<D>;
  constexpr int S = C::kStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const uint32_t sq = ptx::smem_u32(smem + C::kOffQ);
  const uint32_t sk = ptx::smem_u32(smem + C::kOffK);
  const uint32_t sv_ = ptx::smem_u32(smem + C::kOffV);
  const uint32_t bar0 = ptx::smem_u32(smem + C::kOffBar);
  auto BAR = [bar0](int i) -> uint32_t { return bar0 + 8u * (uint32_t)i; };
  auto K_FULL = [&](int st) { return BAR(kKv + st); };
  auto K_EMPTY = [&](int st) { return BAR(kKv + S + st); };
  auto V_FULL = [&](int st) { return BAR(kKv + 2 * S + st); };
  auto V_EMPTY = [&](int st) { return BAR(kKv + 3 * S + st); };
  Misc* misc = reinterpret_cast<Misc*>(smem + C::kOffMisc);
  volatile int* abort_flag = &misc->abort;
  int* err = p.err;
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;

  // ------------------------------------------------------------ work unit
  int idx = blockIdx.x;
  const int pair = idx % p.pairs;
  idx /= p.pairs;
  const int split = idx % p.nsplit;
  const int hkv = idx / p.nsplit;
  const bool has_b = 2 * pair + 1 < p.tiles;
  const int n_x = has_b ? 2 : 1;
  const int n_mma = C::kSepP ? n_x : 1;  // warps issuing MMAs
  const int c0 = split * p.chunk;
  const int key_end = min(c0 + p.chunk, p.Lp);
  const int n_tiles = (key_end - c0 + 127) / 128;  // >= 1
  const bool paged = p.prefix_table != nullptr;

  if (threadIdx.x == 0) {
    ptx::prefetch_tmap(&tm_q);
    ptx::prefetch_tmap(&tm_k);
    ptx::prefetch_tmap(&tm_v);
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::kOffBar);
    for (int x = 0; x < 2; ++x) {
      ptx::mbar_init(&bars[kQFull + x], 1);
      ptx::mbar_init(&bars[kSFull + x], 1);
      ptx::mbar_init(&bars[kSFree + x], 128);
      ptx::mbar_init(&bars[kPFull + x], 128);
      ptx::mbar_init(&bars[kODone + x], 1);
      ptx::mbar_init(&bars[kTurn + x], 128);
    }
    ptx::mbar_init(&bars[kDrain], n_mma);
    for (int st = 0; st < S; ++st) {
      ptx::mbar_init(&bars[kKv + st], 1);
      ptx::mbar_init(&bars[kKv + S + st], n_mma);
      ptx::mbar_init(&bars[kKv + 2 * S + st], 1);
      ptx::mbar_init(&bars[kKv + 3 * S + st], n_mma);
    }
    misc->abort = 0;
    ptx::fence_mbar_init();
  }
  if (warp == 1) {
    ptx::tmem_alloc(&misc->tmem_base, kTmemCols);
    ptx::tmem_relinquish();
  }
  // rows of a Q tile that no box fills: zeros (their results are not stored)
  if (p.box_rows < 128) {
    const int n16 = (128 - p.box_rows) * 8;  // 16-byte pieces per atom
    for (int i = threadIdx.x; i < 2 * C::kAtoms * n16; i += kThreads) {
      const int a = i / n16, o = i - a * n16;
      *reinterpret_cast<uint4*>(smem + C::kOffQ + a * C::kAtomBytes + p.box_rows * 128 + o * 16) =
          make_uint4(0, 0, 0, 0);
    }
    ptx::fence_proxy_async_smem();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = misc->tmem_base;
  // the decode of the sequences' own caches needs nothing from here: it may start as
  // soon as an SM is free
  sched::let_next_kernel_launch();

  if (warp < 4) {
    ptx::regs_dec<kRegsLow>();
    if (warp == 0) {
      // ---------------------------------------------------------- TMA producer
      // Contiguous prefix, or pages of 128 keys or more: one box per 64-column
      // atom.  Shorter pages: one box per page slice and atom, spread over the
      // lanes.  Keys past the prefix read as zeros (out-of-range coordinate);
      // a page id outside the pool does too and flags the error word.
      constexpr uint32_t kTx = C::kTileBytes;
      const int rows = paged && p.page_size < 128 ? p.page_size : 128;  // keys per box
      const int n_items = (128 / rows) * C::kAtoms;                     // at most 16
      const int sub = lane / C::kAtoms, atom = lane % C::kAtoms;
      auto load_kv = [&](uint32_t dst, const CUtensorMap* tm, uint32_t bar, int k0, int z) {
        if (lane == 0) ptx::mbar_arrive_expect_tx_a(bar, kTx);
        __syncwarp();
        if (lane < n_items)
          ptx::tma_load_3d_a(dst + atom * C::kAtomBytes + sub * rows * 128, tm, bar, atom * 64,
                             paged ? (k0 + sub * rows) & (p.page_size - 1) : k0, z);
      };
      // pool index (page * Hkv + hkv) of this lane's box of the tile at k0
      auto pool = [&](int k0) -> int {
        if (!paged) return hkv;
        const int j = k0 + sub * rows;
        if (lane >= n_items || j >= key_end) return -1;
        const int page = __ldg(p.prefix_table + j / p.page_size);
        if (page < 0 || page >= p.num_pages) {
          atomicOr(err, kDevErrBadPage);
          return -1;
        }
        return page * p.Hkv + hkv;
      };
      if (lane == 0) {
        for (int x = 0; x < n_x; ++x) {
          const int tile = 2 * pair + x;
          const int b0 = p.per_seq > 1 ? tile / p.per_seq : tile * p.nb;
          const int y = p.per_seq > 1 ? (tile - b0 * p.per_seq) * 128 : 0;
          ptx::mbar_arrive_expect_tx_a(BAR(kQFull + x), (uint32_t)(p.box_rows * 128 * C::kAtoms));
          for (int a = 0; a < C::kAtoms; ++a)
            tma_load_4d_a(sq + x * C::kTileBytes + a * C::kAtomBytes, &tm_q, BAR(kQFull + x),
                          a * 64, y, hkv, b0);
        }
      }
      int j = 0;
      bool ok = true;
      int z_next = pool(c0);
      for (; j < n_tiles; ++j) {
        const int st = j % S;
        const uint32_t ph = (uint32_t)(j / S) & 1u;
        const int k0 = c0 + j * 128;
        const int z = z_next;
        ok = ptx::mbar_wait_a(K_EMPTY(st), ph ^ 1u, abort_flag, err, kDevErrTimeoutProducer);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        load_kv(sk + st * C::kTileBytes, &tm_k, K_FULL(st), k0, z);
        if (j + 1 < n_tiles) z_next = pool(k0 + 128);  // in flight during the wait
        ok = ptx::mbar_wait_a(V_EMPTY(st), ph ^ 1u, abort_flag, err, kDevErrTimeoutProducer);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        load_kv(sv_ + st * C::kTileBytes, &tm_v, V_FULL(st), k0, z);
      }
      // Drain: every copy lands before the CTA exits (long done in a normal run).
      // After a failed wait, tile j may have its K copy in flight; it was counted
      // on K_FULL like the others.
      if (lane == 0) {
        int dummy = 0;
        for (int x = 0; x < n_x; ++x) {
          dummy = 0;
          ptx::mbar_wait_a(BAR(kQFull + x), 0, &dummy, nullptr, 0);
        }
        for (int jj = max(0, j - S); jj < min(j + (ok ? 0 : 1), n_tiles); ++jj) {
          const uint32_t ph = (uint32_t)(jj / S) & 1u;
          dummy = 0;
          ptx::mbar_wait_a(K_FULL(jj % S), ph, &dummy, nullptr, 0);
          dummy = 0;
          if (jj < j) ptx::mbar_wait_a(V_FULL(jj % S), ph, &dummy, nullptr, 0);
        }
      }
    } else if (warp == 1 || (warp == 2 && n_mma == 2)) {
      // ------------------------------------------------------- MMA issuers
      // The whole warp runs the loop; elect.sync picks the lane that issues.  d = 64:
      // one warp per query tile; d = 128: one for both (with two the 32K-key prefix of 512 rows took 101 us instead of 83).
      constexpr uint32_t kIdescS = ptx::idesc_bf16_f32(128, 128, 0, 0);
      constexpr uint32_t kIdescPV = ptx::idesc_bf16_f32(128, D, 0, 1);
      auto wait = [&](uint32_t bar, uint32_t parity) -> bool {
        const bool w = ptx::mbar_wait_a(bar, parity, abort_flag, err, kDevErrTimeoutMma);
        return __all_sync(0xffffffffu, w);
      };
      auto k_ready = [&](int j) -> bool {
        const bool w = wait(K_FULL(j % S), (uint32_t)(j / S) & 1u);
        ptx::tc_fence_after();
        return w;
      };
      // S_x = Q_x K_j^T; K_j has landed
      auto issue_s = [&](int j, int x) {
        const uint32_t s_tmem = tmem + (x ? 128u : 0u);
        const uint64_t q_desc = ptx::smem_desc_sw128(sq + x * C::kTileBytes, 16, 1024);
        const uint64_t k_desc = ptx::smem_desc_sw128(sk + j % S * C::kTileBytes, 16, 1024);
        if constexpr (D == 64)
          ptx::mma_qk_chain_d64(s_tmem, q_desc, k_desc, kIdescS);
        else
          ptx::mma_qk_chain_d128(s_tmem, q_desc, k_desc, kIdescS);
        ptx::mma_commit_warp(BAR(kSFull + x));
      };
      // O_x += P_x V_j once P_x is written and V_j has landed
      auto issue_pv = [&](int j, int x) -> bool {
        const int st = j % S;
        if (!wait(BAR(kPFull + x), (uint32_t)j & 1u)) return false;
        if (!wait(V_FULL(st), (uint32_t)(j / S) & 1u)) return false;
        ptx::tc_fence_after();
        const uint32_t p_tmem = tmem + (C::kSepP ? 384u + (uint32_t)(x * 64) : x ? 128u : 0u);
        ptx::mma_pv_chain8(tmem + 256u + (uint32_t)(x * D), p_tmem,
                           ptx::smem_desc_sw128(sv_ + st * C::kTileBytes, C::kAtomBytes, 1024),
                           kIdescPV, j > 0 ? 1u : 0u);
        ptx::mma_commit_warp(BAR(kODone + x));
        return true;
      };
      bool ok = true;
      if constexpr (C::kSepP) {
        const int x = warp - 1;
        ok = wait(BAR(kQFull + x), 0) && k_ready(0);
        if (ok) {
          issue_s(0, x);
          ptx::mma_commit_warp(K_EMPTY(0));
        }
        for (int j = 0; j < n_tiles && ok; ++j) {
          // the next S needs S_x loaded; this tile's P V follows when P_x is written
          if (j + 1 < n_tiles) {
            ok = wait(BAR(kSFree + x), (uint32_t)j & 1u) && k_ready(j + 1);
            if (!ok) break;
            issue_s(j + 1, x);
            ptx::mma_commit_warp(K_EMPTY((j + 1) % S));
          }
          ok = issue_pv(j, x);
          if (ok) ptx::mma_commit_warp(V_EMPTY(j % S));
        }
      } else {
        for (int x = 0; x < n_x && ok; ++x) ok = wait(BAR(kQFull + x), 0);
        ok = ok && k_ready(0);
        if (ok) {
          for (int x = 0; x < n_x; ++x) issue_s(0, x);
          ptx::mma_commit_warp(K_EMPTY(0));
        }
        for (int j = 0; j < n_tiles && ok; ++j) {
          for (int x = 0; x < n_x && ok; ++x) {
            // the next S overwrites P_x: right behind this tile's P V, in pipe order
            ok = issue_pv(j, x);
            if (ok && j + 1 < n_tiles) {
              if (x == 0) ok = k_ready(j + 1);
              if (ok) issue_s(j + 1, x);
            }
          }
          if (!ok) break;
          ptx::mma_commit_warp(V_EMPTY(j % S));
          if (j + 1 < n_tiles) ptx::mma_commit_warp(K_EMPTY((j + 1) % S));
        }
      }
      ptx::mma_commit_warp(BAR(kDrain));
      int dummy = 0;
      ptx::mbar_wait_a(BAR(kDrain), 0, &dummy, nullptr, 0);
    }
  } else {
    // ---------------------------------------------------------------- softmax
    ptx::regs_inc<kRegsHigh>();
    const int x = (warp - 4) >> 2;
    if (x < n_x) {
      const int quarter = warp & 3;
      const int r = quarter * 32 + lane;  // row of the tile = TMEM lane
      const uint32_t t_row = tmem + ((uint32_t)(quarter * 32) << 16);
      const uint32_t s_col = x ? 128u : 0u;
      const uint32_t o_col = 256u + (uint32_t)(x * D);
      const uint32_t p_col = C::kSepP ? 384u + (uint32_t)(x * 64) : s_col;
      const float c = p.scale_log2;
      float m_ref = -INFINITY;
      float l = 0.0f;
      bool ok = true;
      if (has_b && x == 1) ptx::mbar_arrive_a(BAR(kTurn));  // B hands A the first turn
      int j = 0;
      for (; j < n_tiles; ++j) {
        const int left = key_end - (c0 + j * 128);  // keys of this tile below the end
        ok = ptx::mbar_wait_a(BAR(kSFull + x), (uint32_t)j & 1u, abort_flag, err,
                              kDevErrTimeoutSoftmax);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        ptx::tc_fence_after();
        float s[128];
        row::tmem_ld_row128(t_row + s_col, s);
        if constexpr (C::kSepP) {
          ptx::tc_fence_before();
          ptx::mbar_arrive_a(BAR(kSFree + x));
        }
        if (left < 128) {
#pragma unroll
          for (int i = 0; i < 128; ++i) s[i] = i < left ? s[i] : -INFINITY;
        }
        const float m_new = fmaxf(m_ref, ptx::row_max128(s) * c);
        const bool need = m_new > m_ref + kRescaleThreshold;
        const float alpha = need ? ptx::ex2(m_ref - m_new) : 1.0f;
        if (need) {
          l *= alpha;
          m_ref = m_new;
        }
        const float m_use = m_ref == -INFINITY ? 0.0f : m_ref;
        if (has_b) {
          ok = ptx::mbar_wait_a(BAR(kTurn + x), (uint32_t)j & 1u, abort_flag, err,
                                kDevErrTimeoutSoftmax);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
        }
        uint32_t pk_lo[32], pk_hi[32];
        l += row::exp2_pack128(s, c, m_use, pk_lo, pk_hi);
        if (has_b) ptx::mbar_arrive_a(BAR(kTurn + (x ^ 1)));
        const bool any_need = __any_sync(0xffffffffu, need);
        if (j > 0 && (C::kSepP || any_need)) {
          // P_x V of the previous tile: done before O_x is rescaled or P_x overwritten
          ok = ptx::mbar_wait_a(BAR(kODone + x), (uint32_t)(j - 1) & 1u, abort_flag, err,
                                kDevErrTimeoutSoftmax);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          ptx::tc_fence_after();
        }
        if (j > 0 && any_need) {
#pragma unroll 1
          for (int cc = 0; cc < D / 32; ++cc) {
            uint32_t raw[32];
            ptx::tmem_ld32(t_row + o_col + cc * 32, raw);
            ptx::tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 32; ++i)
              raw[i] = __float_as_uint(__uint_as_float(raw[i]) * alpha);
            ptx::tmem_st32(t_row + o_col + cc * 32, raw);
          }
        }
        ptx::tmem_st32(t_row + p_col, pk_lo);
        ptx::tmem_st32(t_row + p_col + 32, pk_hi);
        if (paged && left < 128) {
          // V rows of a last page past the prefix may hold anything (even NaN),
          // and 0 * NaN would poison O: zero them.  Both tiles' warpgroups do,
          // each before its own P V.
          const int st = j % S;
          ok = ptx::mbar_wait_a(V_FULL(st), (uint32_t)(j / S) & 1u, abort_flag, err,
                                kDevErrTimeoutSoftmax);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          if (r >= left) {
#pragma unroll
            for (int a = 0; a < C::kAtoms; ++a) {
              uint4* row_ptr = reinterpret_cast<uint4*>(smem + C::kOffV + st * C::kTileBytes +
                                                        a * C::kAtomBytes + r * 128);
#pragma unroll
              for (int q = 0; q < 8; ++q) row_ptr[q] = make_uint4(0, 0, 0, 0);
            }
            ptx::fence_proxy_async_smem();
          }
        }
        ptx::tmem_wait_st();
        ptx::tc_fence_before();
        ptx::mbar_arrive_a(BAR(kPFull + x));
      }
      // ---------------------------------------------------------- epilogue
      if (ok) {
        ok = ptx::mbar_wait_a(BAR(kODone + x), (uint32_t)(n_tiles - 1) & 1u, abort_flag, err,
                              kDevErrTimeoutSoftmax);
        ok = __all_sync(0xffffffffu, ok);
        ptx::tc_fence_after();
      }
      // flat output row of tile row r
      const int tile = 2 * pair + x;
      int b, rr;
      bool row_ok;
      if (p.per_seq > 1) {
        b = tile / p.per_seq;
        rr = (tile - b * p.per_seq) * 128 + r;
        row_ok = rr < p.G;
      } else {
        const int bi = r / p.G;
        b = tile * p.nb + bi;
        rr = r - bi * p.G;
        row_ok = bi < p.nb && b < p.B;
      }
      const long long out = (long long)split * p.nrows + ((long long)b * p.Hkv + hkv) * p.G + rr;
      const bool have = ok && l != 0.0f;  // NaN stays NaN
      const float inv_l = have ? 1.0f / l : 0.0f;
#pragma unroll 1
      for (int cc = 0; cc < D / 32; ++cc) {
        uint32_t raw[32];
        if (ok) {
          ptx::tmem_ld32(t_row + o_col + cc * 32, raw);
          ptx::tmem_wait_ld();
        } else {
#pragma unroll
          for (int i = 0; i < 32; ++i) raw[i] = 0u;
        }
        if (row_ok) {
          float* dst = p.ws_o + out * D + cc * 32;
#pragma unroll
          for (int i = 0; i < 32; i += 4)
            *reinterpret_cast<float4*>(dst + i) = make_float4(
                __uint_as_float(raw[i]) * inv_l, __uint_as_float(raw[i + 1]) * inv_l,
                __uint_as_float(raw[i + 2]) * inv_l, __uint_as_float(raw[i + 3]) * inv_l);
        }
      }
      if (row_ok) p.ws_lse[out] = have ? (m_ref + ptx::lg2(l)) * kLn2 : -INFINITY;
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
cudaError_t launch_prefix(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                          const PrefixParams& p, cudaStream_t stream) {
  auto kern = attn_prefix_kernel<D>;
  constexpr int smem = Cfg<D>::kSmemAlloc;
  static PerContextOnce once;
  const cudaError_t e = once_per_context(once, [&](int) {
    return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  });
  if (e != cudaSuccess) return e;
  const long long grid = (long long)p.Hkv * p.nsplit * p.pairs;
  if (grid > 0x7fffffffLL) return cudaErrorInvalidValue;
  kern<<<(unsigned)grid, kThreads, smem, stream>>>(tq, tk, tv, p);
  return cudaGetLastError();
}

template cudaError_t launch_prefix<64>(const CUtensorMap&, const CUtensorMap&, const CUtensorMap&,
                                       const PrefixParams&, cudaStream_t);
template cudaError_t launch_prefix<128>(const CUtensorMap&, const CUtensorMap&,
                                        const CUtensorMap&, const PrefixParams&, cudaStream_t);

}  // namespace attn
