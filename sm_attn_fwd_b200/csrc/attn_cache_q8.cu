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

template <int D>
__global__ void __launch_bounds__(kCacheThreads) attn_cache_append_kernel(const CacheParams p) {
  constexpr int kLanes = D / 8;
  const long long idx = (long long)blockIdx.x * kCacheThreads + threadIdx.x;
  const int part = threadIdx.x % kLanes;
  const int nrows = p.B * p.Hkv * p.Ln;  // at most 2^31 - 1, checked on the host
  const long long row_l = idx / kLanes;
  bool live = row_l < nrows;
  const int row = live ? (int)row_l : 0;
  const int bh = row / p.Ln, i = row - bh * p.Ln;
  const int b = bh / p.Hkv, h = bh - b * p.Hkv;
  // every lane stays for the shuffles; a lane group is live as a whole
  const int len = __ldg(p.kv_lens + b);
  const int n_new = p.new_lens ? __ldg(p.new_lens + b) : p.Ln;
  if (len < 0 || len > p.Lk || n_new < 0 || n_new > p.Ln || n_new > len) {
    if (live && i == 0 && h == 0 && part == 0) atomicOr(p.err, kDevErrBadKvLen);
    live = false;
  }
  live = live && i < n_new;
  uint4 kr = make_uint4(0, 0, 0, 0), vr = kr;
  if (live) {
    const long long at = (long long)row * kLanes + part;  // in 16-byte units
    kr = __ldcs(reinterpret_cast<const uint4*>(p.k_in) + at);
    vr = __ldcs(reinterpret_cast<const uint4*>(p.v_in) + at);
  }
  const long long dst = live ? cache_row(p, b, h, len - n_new + i) : -1;
  int ek, ev;
  const uint2 kc = quantise8<kLanes>(kr, ek);
  const uint2 vc = quantise8<kLanes>(vr, ev);
  if (dst >= 0) {
    reinterpret_cast<uint2*>(p.k_codes)[dst * kLanes + part] = kc;
    reinterpret_cast<uint2*>(p.v_codes)[dst * kLanes + part] = vc;
    if (part == 0) {
      p.k_exp[dst] = (uint8_t)ek;
      p.v_exp[dst] = (uint8_t)ev;
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

template <int D>
__global__ void __launch_bounds__(kCacheThreads) attn_cache_read_kernel(const CacheParams p) {
  constexpr int kLanes = D / 16;
  const long long idx = (long long)blockIdx.x * kCacheThreads + threadIdx.x;
  const int part = threadIdx.x % kLanes;
  const int nrows = p.B * p.Hkv * p.Lk;
  if (idx / kLanes >= nrows) return;
  const int row = (int)(idx / kLanes);
  const int bh = row / p.Lk, j = row - bh * p.Lk;
  const int b = bh / p.Hkv, h = bh - b * p.Hkv;
  int len = __ldg(p.kv_lens + b);
  if (len < 0 || len > p.Lk) {
    if (j == 0 && h == 0 && part == 0) atomicOr(p.err, kDevErrBadKvLen);
    return;
  }
  if (j >= len) return;
  const long long src = cache_row(p, b, h, j);
  uint4 ko[2], vo[2];
  if (src >= 0) {
    const uint4 kc = __ldcs(reinterpret_cast<const uint4*>(p.k_codes) + src * kLanes + part);
    const uint4 vc = __ldcs(reinterpret_cast<const uint4*>(p.v_codes) + src * kLanes + part);
    restore16(kc, q8::scale_of(p.k_exp[src]), ko);
    restore16(vc, q8::scale_of(p.v_exp[src]), vo);
  } else {
    ko[0] = ko[1] = vo[0] = vo[1] = make_uint4(0, 0, 0, 0);
  }
  const long long dst = ((long long)row * kLanes + part) * 2;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    reinterpret_cast<uint4*>(p.k_out)[dst + i] = ko[i];
    reinterpret_cast<uint4*>(p.v_out)[dst + i] = vo[i];
  }
}

unsigned blocks_for(long long threads) {
  return (unsigned)((threads + kCacheThreads - 1) / kCacheThreads);
}

}  // namespace

template <int D>
cudaError_t launch_cache_append(const CacheParams& p, cudaStream_t stream) {
  const long long rows = (long long)p.B * p.Hkv * p.Ln;
  attn_cache_append_kernel<D><<<blocks_for(rows * (D / 8)), kCacheThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

template <int D>
cudaError_t launch_cache_read(const CacheParams& p, cudaStream_t stream) {
  const long long rows = (long long)p.B * p.Hkv * p.Lk;
  attn_cache_read_kernel<D><<<blocks_for(rows * (D / 16)), kCacheThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

template cudaError_t launch_cache_append<64>(const CacheParams&, cudaStream_t);
template cudaError_t launch_cache_append<128>(const CacheParams&, cudaStream_t);
template cudaError_t launch_cache_read<64>(const CacheParams&, cudaStream_t);
template cudaError_t launch_cache_read<128>(const CacheParams&, cudaStream_t);

}  // namespace attn
