// Writing an 8-bit KV cache and reading it back (format in cache_q8.cuh).
//
// Both kernels are one pass over the rows and bound by memory: append reads
// 2 d bytes and writes d + 1 per row, read-back the reverse.  A row belongs to d / 8
// neighbouring lanes, eight values each: 16 bytes of bf16, 8 of codes, so a warp's
// loads and stores cover whole consecutive rows (read-back with 16 codes per lane
// stored half sectors: 5.1 TB/s instead of 6.7).  The row maximum is a few shuffles
// inside the lane group.  Each lane group handles its K row and its V row together.
//
// Measured against the copy bandwidth of 6.57 TB/s: append of 4 x 8 heads x 8192 tokens,
// d = 128: 30.7 us, 6.6 TB/s; ragged into 64-key pages (126 MB): 24 to 29 us, 4.3 to 5.2
// TB/s; read-back of 16 x 8 heads x 16384 tokens (1.6 GB): 239 us, 6.7 TB/s; one token
// for 64 x 8 heads: 2.0 us, a launch.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "attn_params.h"
#include "cache_q8.cuh"
#include "decode_params.h"
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

// The largest magnitude of eight bf16 values, as its bits (magnitudes of bf16 order
// like their bits; 0x7f80 and above are infinity and NaN).
__device__ __forceinline__ uint32_t max_bits(const uint4& w) {
  const uint32_t m = __vmaxu2(__vmaxu2(w.x & 0x7fff7fffu, w.y & 0x7fff7fffu),
                              __vmaxu2(w.z & 0x7fff7fffu, w.w & 0x7fff7fffu));
  return __vmaxu2(m, m >> 16) & 0xffffu;
}
// The same with infinities and NaN left out: they do not set a row's scale.
__device__ __forceinline__ uint32_t max_finite_bits(const uint4& raw) {
  const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t lo = w[i] & 0x7fffu, hi = (w[i] >> 16) & 0x7fffu;
    if (lo < 0x7f80u) m = max(m, lo);
    if (hi < 0x7f80u) m = max(m, hi);
  }
  return m;
}

// Eight bf16 values times 2^(127 - e) as e4m3 codes.  The product is exact in bf16
// (a power of two; what falls below bf16's range is far below the smallest code).
__device__ __forceinline__ uint2 quantise8(const uint4& raw, int e) {
  const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
  const uint32_t f = (uint32_t)(254 - e) << 7 | (uint32_t)(254 - e) << 23;
  uint32_t c[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 y = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&w[i]),
                                     *reinterpret_cast<const __nv_bfloat162*>(&f));
    const uint32_t b = *reinterpret_cast<const uint32_t*>(&y);
    c[i] = q8::codes2(__uint_as_float(b << 16), __uint_as_float(b & 0xffff0000u));
  }
  return make_uint2(__byte_perm(c[0], c[1], 0x5410), __byte_perm(c[2], c[3], 0x5410));
}

// The kernels were bound by instructions, not memory, as first written (one division
// chain per row, fp32 maxima; 70 % of the issue slots at 1.9 TB/s), so: a block stays
// inside one (sequence, head), whose length and page row it looks up once; the
// maximum of a row runs on packed bf16 magnitudes; K's and V's share their shuffles.
//
// blockIdx.x: chunk of kGroups * U rows; blockIdx.y, z: (b, h).  U rows per lane group,
// kGroups apart: their loads go out together.
template <int D, int U>
__global__ void __launch_bounds__(kCacheThreads) attn_cache_append_kernel(const CacheParams p) {
  constexpr int kLanes = D / 8;
  constexpr int kGroups = kCacheThreads / kLanes;  // rows a block takes at a time
  const int part = threadIdx.x % kLanes;
  const int bh = blockIdx.z * gridDim.y + blockIdx.y;
  if (bh >= p.B * p.Hkv) return;
  const int b = bh / p.Hkv, h = bh - b * p.Hkv;
  const int first = blockIdx.x * (kGroups * U) + threadIdx.x / kLanes;
  const int len = __ldg(p.kv_lens + b);
  const int n_new = p.new_lens ? __ldg(p.new_lens + b) : p.Ln;
  if (len < 0 || len > p.Lk || n_new < 0 || n_new > p.Ln || n_new > len) {
    if (first == 0 && h == 0 && part == 0) atomicOr(p.err, kDevErrBadKvLen);
    return;  // the whole block
  }
  if ((int)blockIdx.x * (kGroups * U) >= n_new) return;
  const long long in0 = (long long)bh * p.Ln * kLanes + part;  // in 16-byte units
  uint4 kr[U], vr[U];
  long long dst[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int i = first + u * kGroups;
    kr[u] = vr[u] = make_uint4(0, 0, 0, 0);
    dst[u] = -1;
    if (i < n_new) {
      kr[u] = __ldcs(reinterpret_cast<const uint4*>(p.k_in) + in0 + (long long)i * kLanes);
      vr[u] = __ldcs(reinterpret_cast<const uint4*>(p.v_in) + in0 + (long long)i * kLanes);
      dst[u] = cache_row(p, b, h, len - n_new + i);
    }
  }
  // every lane takes part in the shuffles; a lane group is live as a whole
#pragma unroll
  for (int u = 0; u < U; ++u) {
    uint32_t m = max_bits(kr[u]) | max_bits(vr[u]) << 16;  // K's maximum, V's maximum
#pragma unroll
    for (int o = kLanes / 2; o > 0; o >>= 1)
      m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, o));
    if (__any_sync(0xffffffffu, (m & 0xffffu) >= 0x7f80u || m >= 0x7f800000u)) {
      m = max_finite_bits(kr[u]) | max_finite_bits(vr[u]) << 16;
#pragma unroll
      for (int o = kLanes / 2; o > 0; o >>= 1)
        m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, o));
    }
    const int ek = q8::scale_byte(__uint_as_float(m << 16));
    const int ev = q8::scale_byte(__uint_as_float(m & 0xffff0000u));
    if (dst[u] >= 0) {
      reinterpret_cast<uint2*>(p.k_codes)[dst[u] * kLanes + part] = quantise8(kr[u], ek);
      reinterpret_cast<uint2*>(p.v_codes)[dst[u] * kLanes + part] = quantise8(vr[u], ev);
      if (part == 0) {
        p.k_exp[dst[u]] = (uint8_t)ek;
        p.v_exp[dst[u]] = (uint8_t)ev;
      }
    }
  }
}

// Eight codes times 2^(e - 127) -> eight bf16 values (16 bytes).  Two codes
// sign-extended into 16-bit halves, shifted by 4 and masked, read as bf16, are the
// values times 2^-120; one packed multiply finishes two of them, exactly except below
// bf16's normal range, where it rounds to nearest even.
__device__ __forceinline__ uint4 restore8(const uint2& c, int e) {
  const uint32_t w[2] = {c.x, c.y};
  uint32_t r[4];
  // 2^(e - 7); above bf16's range (e > 134) 2^120 and 2^(e - 127) one after the other
  const uint32_t x = e <= 134 ? (uint32_t)(e + 120) : 247u;
  const uint32_t f = x << 7 | x << 23;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t v;
    asm("prmt.b32 %0, %1, 0, %2;" : "=r"(v) : "r"(w[i >> 1]), "r"(i & 1 ? 0xb3a2 : 0x9180));
    v = (v << 4) & 0x87f087f0u;
    const __nv_bfloat162 y = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&v),
                                     *reinterpret_cast<const __nv_bfloat162*>(&f));
    r[i] = *reinterpret_cast<const uint32_t*>(&y);
  }
  if (e > 134) {
    const uint32_t x2 = (uint32_t)min(e, q8::kMaxScaleByte), f2 = x2 << 7 | x2 << 23;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 y = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&r[i]),
                                       *reinterpret_cast<const __nv_bfloat162*>(&f2));
      r[i] = *reinterpret_cast<const uint32_t*>(&y);
    }
  }
  // NaN codes (magnitude 0x7f) come back as NaN: a carry out of a byte marks them
  if ((((w[0] & 0x7f7f7f7fu) + 0x01010101u) | ((w[1] & 0x7f7f7f7fu) + 0x01010101u)) &
      0x80808080u) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (((w[i >> 2] >> (8 * (i & 3))) & 0x7fu) == 0x7fu) r[i >> 1] |= 0x7fffu << (16 * (i & 1));
  }
  return make_uint4(r[0], r[1], r[2], r[3]);
}

template <int D, int U>
__global__ void __launch_bounds__(kCacheThreads) attn_cache_read_kernel(const CacheParams p) {
  constexpr int kLanes = D / 8;
  constexpr int kGroups = kCacheThreads / kLanes;
  const int part = threadIdx.x % kLanes;
  const int bh = blockIdx.z * gridDim.y + blockIdx.y;
  if (bh >= p.B * p.Hkv) return;
  const int b = bh / p.Hkv, h = bh - b * p.Hkv;
  const int first = blockIdx.x * (kGroups * U) + threadIdx.x / kLanes;
  const int len = __ldg(p.kv_lens + b);
  if (len < 0 || len > p.Lk) {
    if (first == 0 && h == 0 && part == 0) atomicOr(p.err, kDevErrBadKvLen);
    return;
  }
  uint2 kc[U], vc[U];
  int ke[U], ve[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int j = first + u * kGroups;
    kc[u] = vc[u] = make_uint2(0, 0);
    ke[u] = ve[u] = 1;
    if (j >= len) continue;
    const long long src = cache_row(p, b, h, j);
    if (src < 0) continue;  // reads as zeros
    kc[u] = __ldcs(reinterpret_cast<const uint2*>(p.k_codes) + src * kLanes + part);
    vc[u] = __ldcs(reinterpret_cast<const uint2*>(p.v_codes) + src * kLanes + part);
    ke[u] = __ldg(p.k_exp + src);
    ve[u] = __ldg(p.v_exp + src);
  }
  const long long out0 = (long long)bh * p.Lk * kLanes + part;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int j = first + u * kGroups;
    if (j >= len) continue;
    const long long dst = out0 + (long long)j * kLanes;
    __stcs(reinterpret_cast<uint4*>(p.k_out) + dst, restore8(kc[u], ke[u]));
    __stcs(reinterpret_cast<uint4*>(p.v_out) + dst, restore8(vc[u], ve[u]));
  }
}

// Rows per lane group: four once a launch has more rows than the device holds threads
// for (2048 per SM) anyway, so that a thread has several loads in flight; with fewer
// rows that would leave SMs idle.  Four against one, us: read-back of 8 x 8 heads, up to
// 32768 tokens: 158 / 178; append of 4 x 8 heads, up to 8192: 24.2 / 25.9; below the
// limit, append of 7 x 4 heads, up to 2064: 5.7 / 5.3; one token for 64 x 8 heads:
// 3.2 / 2.0; read-back of 5 x 4 heads, up to 2064: 4.5 / 3.9.
constexpr int kRowsPerGroup = 4;
bool many_rows(long long rows, int lanes, int num_sms) {
  return rows * lanes > 2LL * num_sms * 2048;
}

// Chunks of `rows` rows by (b, h) pairs, the pairs in y and z (each at most 65535).
dim3 cache_grid(int rows, int lanes, int u, long long pairs) {
  const int per = kCacheThreads / lanes * u;
  const long long y = pairs < 65535 ? pairs : 65535;
  return dim3((unsigned)((rows + (long long)per - 1) / per), (unsigned)y,
              (unsigned)((pairs + y - 1) / y));
}

}  // namespace

template <int D>
cudaError_t launch_cache_append(const CacheParams& p, int num_sms, cudaStream_t stream) {
  constexpr int kLanes = D / 8, U = kRowsPerGroup;
  const long long pairs = (long long)p.B * p.Hkv;
  if (many_rows(pairs * p.Ln, kLanes, num_sms))
    attn_cache_append_kernel<D, U>
        <<<cache_grid(p.Ln, kLanes, U, pairs), kCacheThreads, 0, stream>>>(p);
  else
    attn_cache_append_kernel<D, 1>
        <<<cache_grid(p.Ln, kLanes, 1, pairs), kCacheThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

template <int D>
cudaError_t launch_cache_read(const CacheParams& p, int num_sms, cudaStream_t stream) {
  constexpr int kLanes = D / 8, U = kRowsPerGroup;
  const long long pairs = (long long)p.B * p.Hkv;
  if (many_rows(pairs * p.Lk, kLanes, num_sms))
    attn_cache_read_kernel<D, U>
        <<<cache_grid(p.Lk, kLanes, U, pairs), kCacheThreads, 0, stream>>>(p);
  else
    attn_cache_read_kernel<D, 1>
        <<<cache_grid(p.Lk, kLanes, 1, pairs), kCacheThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

template cudaError_t launch_cache_append<64>(const CacheParams&, int, cudaStream_t);
template cudaError_t launch_cache_append<128>(const CacheParams&, int, cudaStream_t);
template cudaError_t launch_cache_read<64>(const CacheParams&, int, cudaStream_t);
template cudaError_t launch_cache_read<128>(const CacheParams&, int, cudaStream_t);

}  // namespace attn
