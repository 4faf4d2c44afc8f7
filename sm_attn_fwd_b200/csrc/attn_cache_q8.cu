// Writing an 8-bit KV cache and reading it back (format in cache_q8.cuh).
//
// Both kernels are one pass over the rows and bound by memory: append reads
// 2 d bytes and writes d + 1 per row, read-back the reverse.  A row belongs to
// d / 8 neighbouring lanes (append: 8 bf16 values, one 16-byte load each) or
// d / 16 (read-back: 16 codes, one 16-byte load each), so a warp's accesses cover
// whole consecutive rows; the row maximum is a few shuffles inside the lane
// group.  Each lane group handles its K row and its V row together, two loads in
// flight per thread.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "attn_params.h"
#include "cache_q8.cuh"
#include "cache_q8_params.h"
#include "ptx.cuh"

namespace attn {
namespace {

constexpr int kCacheThreads = 256;

// Row of the cache (codes at row * d, scale byte at row) that holds key j of
// (b, h); -1 for a page id outside the pool, which flags the error word.
__device__ __forceinline__ long long cache_row(const CacheParams& p, int b, int h, int j) {
  if (p.block_table == nullptr) return ((long long)b * p.Hkv + h) * p.Lk + j;
  const int page = __ldg(p.block_table + (long long)b * p.pages_per_seq + (j >> p.page_shift));
  if (page < 0 || page >= p.num_pages) {
    atomicOr(p.err, kDevErrBadPage);
    return -1;
  }
  return (((long long)page * p.Hkv + h) << p.page_shift) + (j & ((1 << p.page_shift) - 1));
}

// Eight bf16 values (one 16-byte load) of a row shared by kLanes lanes -> their codes.
template <int kLanes>
__device__ __forceinline__ uint2 quantise8(const uint4& raw, int& e_out) {
  const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
  float x[8];
  float amax = 0.0f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    // infinities and NaN do not set the scale (fmaxf drops NaN): an infinity saturates
    const float a = fabsf(x[i]);
    amax = fmaxf(amax, a < INFINITY ? a : 0.0f);
  }
#pragma unroll
  for (int o = kLanes / 2; o > 0; o >>= 1)
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  const int e = q8::scale_byte(amax);
  const float inv = q8::inv_scale_of(e);
  e_out = e;
  uint2 c;
  c.x = q8::codes2(x[0] * inv, x[1] * inv) | (q8::codes2(x[2] * inv, x[3] * inv) << 16);
  c.y = q8::codes2(x[4] * inv, x[5] * inv) | (q8::codes2(x[6] * inv, x[7] * inv) << 16);
  return c;
}

// U rows per lane group, kCacheThreads / kLanes rows apart: their loads go out together.
template <int D, int U>
__global__ void __launch_bounds__(kCacheThreads) attn_cache_append_kernel(const CacheParams p) {
  constexpr int kLanes = D / 8;
  constexpr int kGroups = kCacheThreads / kLanes;  // rows a block takes at a time
  const int part = threadIdx.x % kLanes;
  const int nrows = p.B * p.Hkv * p.Ln;  // at most 2^31 - 1, checked on the host
  const long long first = (long long)blockIdx.x * (kGroups * U) + threadIdx.x / kLanes;
  uint4 kr[U], vr[U];
  long long dst[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    kr[u] = vr[u] = make_uint4(0, 0, 0, 0);
    dst[u] = -1;
    if (first + u * kGroups >= nrows) continue;
    const int row = (int)(first + u * kGroups);
    const int bh = row / p.Ln, i = row - bh * p.Ln;
    const int b = bh / p.Hkv, h = bh - b * p.Hkv;
    const int len = __ldg(p.kv_lens + b);
    const int n_new = p.new_lens ? __ldg(p.new_lens + b) : p.Ln;
    if (len < 0 || len > p.Lk || n_new < 0 || n_new > p.Ln || n_new > len) {
      if (i == 0 && h == 0 && part == 0) atomicOr(p.err, kDevErrBadKvLen);
      continue;
    }
    if (i >= n_new) continue;
    const long long at = (long long)row * kLanes + part;  // in 16-byte units
    kr[u] = __ldcs(reinterpret_cast<const uint4*>(p.k_in) + at);
    vr[u] = __ldcs(reinterpret_cast<const uint4*>(p.v_in) + at);
    dst[u] = cache_row(p, b, h, len - n_new + i);
  }
  // every lane takes part in the shuffles; a lane group is live as a whole
#pragma unroll
  for (int u = 0; u < U; ++u) {
    int ek, ev;
    const uint2 kc = quantise8<kLanes>(kr[u], ek);
    const uint2 vc = quantise8<kLanes>(vr[u], ev);
    if (dst[u] >= 0) {
      reinterpret_cast<uint2*>(p.k_codes)[dst[u] * kLanes + part] = kc;
      reinterpret_cast<uint2*>(p.v_codes)[dst[u] * kLanes + part] = vc;
      if (part == 0) {
        p.k_exp[dst[u]] = (uint8_t)ek;
        p.v_exp[dst[u]] = (uint8_t)ev;
      }
    }
  }
}

// 16 codes times 2^(e - 127) -> 16 bf16 values (32 bytes).  code * scale is exact
// in fp32, so the only rounding is to bf16, and it rounds only below bf16's
// normal range (a code has 4 significant bits).
__device__ __forceinline__ void restore16(const uint4& c, float s, uint4 (&out)[2]) {
  const uint32_t w[4] = {c.x, c.y, c.z, c.w};
  uint32_t r[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t lo, hi;
    q8::codes4_to_f16(w[i], lo, hi);
    const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&lo));
    const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&hi));
    r[2 * i] = ptx::pack_bf16x2(a.x * s, a.y * s);
    r[2 * i + 1] = ptx::pack_bf16x2(b.x * s, b.y * s);
  }
  out[0] = make_uint4(r[0], r[1], r[2], r[3]);
  out[1] = make_uint4(r[4], r[5], r[6], r[7]);
}

template <int D, int U>
__global__ void __launch_bounds__(kCacheThreads) attn_cache_read_kernel(const CacheParams p) {
  constexpr int kLanes = D / 16;
  constexpr int kGroups = kCacheThreads / kLanes;
  const int part = threadIdx.x % kLanes;
  const int nrows = p.B * p.Hkv * p.Lk;
  const long long first = (long long)blockIdx.x * (kGroups * U) + threadIdx.x / kLanes;
  uint4 kc[U], vc[U];
  float ks[U], vs[U];
  bool live[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    kc[u] = vc[u] = make_uint4(0, 0, 0, 0);
    ks[u] = vs[u] = 0.0f;
    live[u] = false;
    if (first + u * kGroups >= nrows) continue;
    const int row = (int)(first + u * kGroups);
    const int bh = row / p.Lk, j = row - bh * p.Lk;
    const int b = bh / p.Hkv, h = bh - b * p.Hkv;
    const int len = __ldg(p.kv_lens + b);
    if (len < 0 || len > p.Lk) {
      if (j == 0 && h == 0 && part == 0) atomicOr(p.err, kDevErrBadKvLen);
      continue;
    }
    if (j >= len) continue;
    live[u] = true;
    const long long src = cache_row(p, b, h, j);
    if (src < 0) continue;  // reads as zeros
    kc[u] = __ldcs(reinterpret_cast<const uint4*>(p.k_codes) + src * kLanes + part);
    vc[u] = __ldcs(reinterpret_cast<const uint4*>(p.v_codes) + src * kLanes + part);
    ks[u] = q8::scale_of(__ldg(p.k_exp + src));
    vs[u] = q8::scale_of(__ldg(p.v_exp + src));
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    if (!live[u]) continue;
    uint4 ko[2], vo[2];
    restore16(kc[u], ks[u], ko);
    restore16(vc[u], vs[u], vo);
    const long long dst = ((first + u * kGroups) * kLanes + part) * 2;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      __stcs(reinterpret_cast<uint4*>(p.k_out) + dst + i, ko[i]);
      __stcs(reinterpret_cast<uint4*>(p.v_out) + dst + i, vo[i]);
    }
  }
}

// Rows per lane group: several once a launch has more rows than the device holds
// threads for (2048 per SM) anyway.
constexpr int kRowsPerGroup = 4;
bool many_rows(long long rows, int lanes) { return rows * lanes > 2LL * 148 * 2048; }

unsigned blocks_for(long long rows, int lanes, int u) {
  const long long per = (long long)(kCacheThreads / lanes) * u;
  return (unsigned)((rows + per - 1) / per);
}

}  // namespace

template <int D>
cudaError_t launch_cache_append(const CacheParams& p, cudaStream_t stream) {
  constexpr int kLanes = D / 8, U = kRowsPerGroup;
  const long long rows = (long long)p.B * p.Hkv * p.Ln;
  if (many_rows(rows, kLanes))
    attn_cache_append_kernel<D, U><<<blocks_for(rows, kLanes, U), kCacheThreads, 0, stream>>>(p);
  else
    attn_cache_append_kernel<D, 1><<<blocks_for(rows, kLanes, 1), kCacheThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

template <int D>
cudaError_t launch_cache_read(const CacheParams& p, cudaStream_t stream) {
  constexpr int kLanes = D / 16, U = kRowsPerGroup;
  const long long rows = (long long)p.B * p.Hkv * p.Lk;
  if (many_rows(rows, kLanes))
    attn_cache_read_kernel<D, U><<<blocks_for(rows, kLanes, U), kCacheThreads, 0, stream>>>(p);
  else
    attn_cache_read_kernel<D, 1><<<blocks_for(rows, kLanes, 1), kCacheThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

template cudaError_t launch_cache_append<64>(const CacheParams&, cudaStream_t);
template cudaError_t launch_cache_append<128>(const CacheParams&, cudaStream_t);
template cudaError_t launch_cache_read<64>(const CacheParams&, cudaStream_t);
template cudaError_t launch_cache_read<128>(const CacheParams&, cudaStream_t);

}  // namespace attn
