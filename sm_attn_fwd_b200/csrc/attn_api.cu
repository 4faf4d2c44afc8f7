// Host side of the C ABI declared in include/attn.h: argument validation,
// split planning, TMA tensor-map encoding and kernel launches.  Nothing here
// allocates device memory or synchronises, except attn_get_device_error.
#include <cuda.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <mutex>

#include "attn.h"
#include "attn_bwd_params.h"
#include "attn_params.h"
#include "attn_prefix_params.h"
#include "decode_params.h"
#include "host_once.h"

namespace attn {
template <int D>
cudaError_t launch_decode(const CUtensorMap&, const CUtensorMap&, const CUtensorMap&,
                          const FwdParams&, dim3, cudaStream_t);
template <int D>
cudaError_t launch_combine(const FwdParams&, cudaStream_t);
template <int D>
cudaError_t launch_prefill(const CUtensorMap&, const CUtensorMap&, const CUtensorMap&,
                           const FwdParams&, int, cudaStream_t);

int* device_error_word();
template <int D>
cudaError_t launch_backward(const CUtensorMap&, const CUtensorMap&, const CUtensorMap&,
                            const CUtensorMap&, const CUtensorMap&, const BwdParams&,
                            cudaStream_t);
cudaError_t launch_selftest_wait(cudaStream_t stream);
template <int D>
cudaError_t launch_short(const CUtensorMap&, const CUtensorMap&, const CUtensorMap&,
                         const FwdParams&, int, cudaStream_t);
template <int D>
cudaError_t launch_cache_append(const CacheParams&, int num_sms, cudaStream_t);
template <int D>
cudaError_t launch_cache_read(const CacheParams&, int num_sms, cudaStream_t);
template <int D, bool kQ8>
cudaError_t launch_decode_rows(const CUtensorMap&, const CUtensorMap&, const DecodeParams&,
                               cudaStream_t);
int decode_rows_box(int d, bool q8, int page_size);
template <int D>
cudaError_t launch_decode_q8_wide(const CUtensorMap&, const CUtensorMap&, const CUtensorMap&,
                                  const DecodeParams&, cudaStream_t);
template <int D>
cudaError_t launch_decode_merge(const DecodeParams&, int num_sms, cudaStream_t);
template <int D>
cudaError_t launch_prefix(const CUtensorMap&, const CUtensorMap&, const CUtensorMap&,
                          const PrefixParams&, cudaStream_t);
}  // namespace attn

namespace {

using attn::FwdParams;
using attn::kBlockM;
using attn::kBlockN;

constexpr long long kMaxGridY = 65535;

PFN_cuTensorMapEncodeTiled_v12000 get_encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* ptr = nullptr;
    cudaDriverEntryPointQueryResult qres;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &ptr, cudaEnableDefault, &qres) ==
            cudaSuccess &&
        qres == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
  });
  return fn;
}

}  // namespace

unsigned long long attn::current_context_id() {
  static PFN_cuCtxGetCurrent_v4000 get_current = nullptr;
  static PFN_cuCtxGetId_v12000 get_id = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* ptr = nullptr;
    cudaDriverEntryPointQueryResult qres;
    if (cudaGetDriverEntryPoint("cuCtxGetCurrent", &ptr, cudaEnableDefault, &qres) ==
            cudaSuccess &&
        qres == cudaDriverEntryPointSuccess)
      get_current = reinterpret_cast<PFN_cuCtxGetCurrent_v4000>(ptr);
    ptr = nullptr;
    if (cudaGetDriverEntryPoint("cuCtxGetId", &ptr, cudaEnableDefault, &qres) == cudaSuccess &&
        qres == cudaDriverEntryPointSuccess)
      get_id = reinterpret_cast<PFN_cuCtxGetId_v12000>(ptr);
  });
  if (!get_current || !get_id) return 0;
  CUcontext ctx = nullptr;
  if (get_current(&ctx) != CUDA_SUCCESS || ctx == nullptr) return 0;
  unsigned long long id = 0;
  if (get_id(ctx, &id) != CUDA_SUCCESS) return 0;
  return id;
}

namespace {

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// Encoded tensor maps are a pure function of their arguments; a small
// per-thread cache skips the encode (a driver call) when a caller repeats a
// call on the same buffers and shapes, as decode and training loops do.
struct TmapKey {
  const void* base;
  uint64_t dims[3];
  int rank, box_rows, kind;
  uint64_t dim3 = 0;  // fourth dimension
  bool operator==(const TmapKey& o) const {
    return base == o.base && rank == o.rank && box_rows == o.box_rows && kind == o.kind &&
           dims[0] == o.dims[0] && dims[1] == o.dims[1] && dims[2] == o.dims[2] &&
           dim3 == o.dim3;
  }
};
constexpr int kTmapCacheSize = 64;
struct TmapCache {
  TmapKey key[kTmapCacheSize];
  CUtensorMap map[kTmapCacheSize];
  bool valid[kTmapCacheSize] = {};
  int next = 0;
};
thread_local TmapCache t_tmaps;

template <class Encode>
bool cached_encode(CUtensorMap* map, const TmapKey& key, Encode&& encode) {
  for (int i = 0; i < kTmapCacheSize; ++i) {
    if (t_tmaps.valid[i] && t_tmaps.key[i] == key) {
      *map = t_tmaps.map[i];
      return true;
    }
  }
  if (!encode(map)) return false;
  const int slot = t_tmaps.next;
  t_tmaps.next = (slot + 1) % kTmapCacheSize;
  t_tmaps.key[slot] = key;
  t_tmaps.map[slot] = *map;
  t_tmaps.valid[slot] = true;
  return true;
}

// bf16 tensor map of rank 2 or 3 (innermost first), boxes of 64 columns by
// box_rows rows, 128-byte swizzle; out-of-range rows read as zero.
bool encode_bf16(CUtensorMap* map, const void* base, int rank, const uint64_t* dims,
                 int box_rows = kBlockN) {
  TmapKey key{base, {dims[0], rank > 1 ? dims[1] : 0, rank > 2 ? dims[2] : 0}, rank, box_rows, 0};
  return cached_encode(map, key, [&](CUtensorMap* out) {
    auto fn = get_encode_fn();
    if (!fn) return false;
    cuuint64_t gdim[3];
    cuuint64_t gstride[2];
    cuuint32_t box[3] = {64, (cuuint32_t)box_rows, 1};
    cuuint32_t estride[3] = {1, 1, 1};
    uint64_t stride = 2;
    for (int i = 0; i < rank; ++i) {
      gdim[i] = dims[i];
      if (i > 0) gstride[i - 1] = stride;
      stride *= dims[i];
    }
    CUresult r = fn(out, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, (cuuint32_t)rank,
                    const_cast<void*>(base), gdim, gstride, box, estride,
                    CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                    CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS;
  });
}

// fp32 tensor of rank 3 {cols, rows, planes} for bulk reduce-adds from shared
// memory: boxes of 32 columns (128 bytes) by 128 rows, 128-byte swizzle.
bool encode_f32_reduce(CUtensorMap* map, const void* base, const uint64_t* dims) {
  TmapKey key{base, {dims[0], dims[1], dims[2]}, 3, kBlockN, 2};
  return cached_encode(map, key, [&](CUtensorMap* out) {
    auto fn = get_encode_fn();
    if (!fn) return false;
    cuuint64_t gdim[3] = {dims[0], dims[1], dims[2]};
    cuuint64_t gstride[2] = {dims[0] * 4, dims[0] * dims[1] * 4};
    cuuint32_t box[3] = {32, (cuuint32_t)kBlockN, 1};
    cuuint32_t estride[3] = {1, 1, 1};
    CUresult r = fn(out, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 3u, const_cast<void*>(base), gdim,
                    gstride, box, estride, CU_TENSOR_MAP_INTERLEAVE_NONE,
                    CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                    CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS;
  });
}

// Token-major packed tensor [total, H, d]: dims {d, H, total}, one head per
// box row group: box {64 columns, 1 head, 128 tokens}, the same shared-memory
// image as a 128-row box of the [B, H, L, d] layout.
bool encode_bf16_packed(CUtensorMap* map, const void* base, int d, int H, int total) {
  TmapKey key{base, {(uint64_t)d, (uint64_t)H, (uint64_t)total}, 3, kBlockN, 1};
  return cached_encode(map, key, [&](CUtensorMap* out) {
    auto fn = get_encode_fn();
    if (!fn) return false;
    cuuint64_t gdim[3] = {(cuuint64_t)d, (cuuint64_t)H, (cuuint64_t)total};
    cuuint64_t gstride[2] = {(cuuint64_t)d * 2, (cuuint64_t)H * d * 2};
    cuuint32_t box[3] = {64, 1, (cuuint32_t)kBlockN};
    cuuint32_t estride[3] = {1, 1, 1};
    CUresult r = fn(out, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3u, const_cast<void*>(base), gdim,
                    gstride, box, estride, CU_TENSOR_MAP_INTERLEAVE_NONE,
                    CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                    CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS;
  });
}

// Query rows of a KV head across sequences: q [B, Hkv, G, d] as {d, G, Hkv, B},
// boxes of 64 columns by box_g rows of one head of box_b sequences (rows of
// consecutive sequences land one after another).
bool encode_bf16_rows(CUtensorMap* map, const void* base, int d, int G, int Hkv, int B, int box_g,
                      int box_b) {
  TmapKey key{base, {(uint64_t)d, (uint64_t)G, (uint64_t)Hkv}, 4, box_g * 256 + box_b, 4,
              (uint64_t)B};
  return cached_encode(map, key, [&](CUtensorMap* out) {
    auto fn = get_encode_fn();
    if (!fn) return false;
    cuuint64_t gdim[4] = {(cuuint64_t)d, (cuuint64_t)G, (cuuint64_t)Hkv, (cuuint64_t)B};
    cuuint64_t row = (cuuint64_t)d * 2;
    cuuint64_t gstride[3] = {row, row * G, row * G * Hkv};
    cuuint32_t box[4] = {64, (cuuint32_t)box_g, 1, (cuuint32_t)box_b};
    cuuint32_t estride[4] = {1, 1, 1, 1};
    CUresult r = fn(out, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4u, const_cast<void*>(base), gdim,
                    gstride, box, estride, CU_TENSOR_MAP_INTERLEAVE_NONE,
                    CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                    CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS;
  });
}

// 8-bit codes {d, rows, planes}: boxes of a whole row (d = 64 or 128 bytes) by
// box_rows rows, swizzled over the row's width; out-of-range rows read as zero.
bool encode_codes(CUtensorMap* map, const void* base, const uint64_t* dims, int box_rows) {
  TmapKey key{base, {dims[0], dims[1], dims[2]}, 3, box_rows, 3};
  return cached_encode(map, key, [&](CUtensorMap* out) {
    auto fn = get_encode_fn();
    if (!fn) return false;
    cuuint64_t gdim[3] = {dims[0], dims[1], dims[2]};
    cuuint64_t gstride[2] = {dims[0], dims[0] * dims[1]};
    cuuint32_t box[3] = {(cuuint32_t)dims[0], (cuuint32_t)box_rows, 1};
    cuuint32_t estride[3] = {1, 1, 1};
    CUresult r = fn(out, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3u, const_cast<void*>(base), gdim, gstride,
                    box, estride, CU_TENSOR_MAP_INTERLEAVE_NONE,
                    dims[0] == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                    CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS;
  });
}

// SM count of the current device (148 when no device answers), queried once
// per device and thread.
int num_sms() {
  thread_local int cached[attn::kMaxDevices] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= attn::kMaxDevices) return 148;
  if (cached[dev] == 0) {
    int v = 0;
    if (cudaDeviceGetAttribute(&v, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || v <= 0)
      return 148;
    cached[dev] = v;
  }
  return cached[dev];
}

long long ceil_div(long long a, long long b) { return (a + b - 1) / b; }

// Device address of the kernels' error word, looked up once per device and
// context.
int* error_word_for_current_device() {
  static attn::PerContextOnce once;
  static int* cache[attn::kMaxDevices] = {};
  int* out = nullptr;
  const cudaError_t e = attn::once_per_context(once, [&](int dev) {
    cache[dev] = attn::device_error_word();
    return cache[dev] ? cudaSuccess : cudaErrorInvalidSymbol;
  });
  if (e != cudaSuccess) return nullptr;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return nullptr;
  std::lock_guard<std::mutex> lock(once.mu);
  out = cache[dev];
  return out;
}

struct SplitPlan {
  int nsplit;
  int chunk;
  int row_tiles;
};

// Returns false for invalid shape arguments.
bool plan_splits(int B, int Hq, int Hkv, int Lq, int Lk_max, int d, int num_splits,
                 SplitPlan* plan) {
  if (B < 1 || Hq < 1 || Hkv < 1 || Lq < 1 || Lk_max < 1 || d < 1 || num_splits < 0) return false;
  if (Hq % Hkv) return false;
  const long long group = Hq / Hkv;
  const long long row_tiles = ceil_div(group * Lq, kBlockM);
  const long long max_splits = ceil_div(Lk_max, kBlockN);
  long long splits;
  if (num_splits > 0) {
    splits = num_splits < max_splits ? num_splits : max_splits;
  } else {
    // At least two waves of CTAs over the SMs, and chunks of at most 12288 keys
    // so that ragged per-sequence lengths balance across the grid.  Shorter
    // chunks cost more than they balance: each split CTA pays a fixed start
    // (Q load, pipeline fill) and end (epilogue, its partial rows written here
    // and read back by the combine, 512 bytes per query row and split).
    const long long units = (long long)B * Hkv * row_tiles;
    long long want = ceil_div(2LL * num_sms(), units);
    const long long by_len = ceil_div(Lk_max, 12288);
    if (by_len > want) want = by_len;
    splits = want < max_splits ? want : max_splits;
  }
  const long long chunk = ceil_div(ceil_div(Lk_max, splits), kBlockN) * kBlockN;
  plan->chunk = (int)chunk;
  plan->nsplit = (int)ceil_div(Lk_max, chunk);
  plan->row_tiles = (int)row_tiles;
  return true;
}

size_t ws_lse_offset(const SplitPlan& pl, long long nrows, int d) {
  const size_t obytes = (size_t)pl.nsplit * (size_t)nrows * (size_t)d * 4;
  return (obytes + 255) / 256 * 256;
}

}  // namespace

namespace {

// Short-query plan: taken when Lq <= 128, the row tiles of all (b, kv head)
// are fewer than twice the SM count, and the key range that any query row can
// see under the mask (before document ids; the lower and upper bounds of a
// row's interval never decrease with its position) spans at least 4 key tiles.
// The cluster of a row tile splits that range into `cluster` chunks of whole
// 128-key tiles, at most 8 CTAs per cluster and at least 8 tiles per CTA.
struct ShortPlan {
  int row_tiles, units, key_lo, chunk, cluster;
};

bool plan_short(int B, int Hq, int Hkv, int Lq, int Lk, int mask_kind, int wl, int wr, int bd,
                ShortPlan* sp) {
  if (Lq > kBlockM) return false;
  const long long group = Hq / Hkv;
  const long long row_tiles = ceil_div(group * Lq, kBlockM);
  const long long units = (long long)B * Hkv * row_tiles;
  const int sms = num_sms();
  if (units >= 2LL * sms || units > kMaxGridY) return false;
  // union of the rows' key intervals: positions Lk - Lq .. Lk - 1
  const long long p_lo = (long long)Lk - Lq, p_hi = (long long)Lk - 1;
  long long lo = 0, hi = (long long)Lk - 1;
  if (mask_kind == ATTN_MASK_CAUSAL) {
    hi = std::min(hi, p_hi);
  } else if (mask_kind == ATTN_MASK_DRAFT_BLOCK) {
    const long long blk = p_hi >= 0 ? p_hi / bd : -((-p_hi + bd - 1) / bd);
    hi = std::min(hi, (blk + 1) * bd - 1);
  }
  if (wl >= 0) lo = std::max(lo, p_lo - wl);
  if (wr >= 0) hi = std::min(hi, p_hi + wr);
  if (hi < lo) return false;  // no row sees a key: the persistent kernel writes the empty rows
  const long long t0 = lo / kBlockN, t1 = hi / kBlockN;
  const long long tiles = t1 - t0 + 1;
  // A few tiles per head are cheaper in the persistent kernel.  A cluster CTA
  // costs several microseconds of start-up and cold loads, so the key range is
  // split only into chunks of at least kMinTilesPerCta tiles.
  constexpr long long kMinTiles = 4, kMinTilesPerCta = 8;
  if (tiles < kMinTiles) return false;
  long long cluster = std::min<long long>(8, ceil_div(2LL * sms, units));
  cluster = std::max<long long>(1, std::min(cluster, tiles / kMinTilesPerCta));
  const long long per = ceil_div(tiles, cluster);
  cluster = ceil_div(tiles, per);
  sp->row_tiles = (int)row_tiles;
  sp->units = (int)units;
  sp->key_lo = (int)(t0 * kBlockN);
  sp->chunk = (int)(per * kBlockN);
  sp->cluster = (int)cluster;
  return true;
}

bool plan_short_possible(int B, int Hq, int Hkv, int Lq, int Lk, int mask_kind, int wl, int wr,
                         int draft_block) {
  ShortPlan sp;
  return plan_short(B, Hq, Hkv, Lq, Lk, mask_kind, wl, wr,
                    mask_kind == ATTN_MASK_DRAFT_BLOCK ? draft_block : 1, &sp);
}

}  // namespace

extern "C" {

const char* attn_status_string(attn_status_t s) {
  switch (s) {
    case ATTN_OK: return "ATTN_OK";
    case ATTN_ERR_INVALID_ARG: return "ATTN_ERR_INVALID_ARG";
    case ATTN_ERR_UNSUPPORTED: return "ATTN_ERR_UNSUPPORTED";
    case ATTN_ERR_WORKSPACE: return "ATTN_ERR_WORKSPACE";
    case ATTN_ERR_CUDA: return "ATTN_ERR_CUDA";
    case ATTN_ERR_TIMEOUT: return "ATTN_ERR_TIMEOUT";
  }
  return "ATTN_ERR_UNKNOWN";
}

// Score modifier of a call (ALiBi slopes or a relative-position table; at most one).
struct ScoreMod {
  const float* alibi_slopes = nullptr;
  const float* rel_table = nullptr;
  int rel_max = 0;
};

// Checks the score_mod arguments of the *_score_mod entry points.
static attn_status_t parse_score_mod(int kind, const float* params, int arg, ScoreMod* sm) {
  *sm = ScoreMod{};
  if (kind == ATTN_SCORE_MOD_NONE) return ATTN_OK;
  if (!params || !aligned(params, 4)) return ATTN_ERR_INVALID_ARG;
  if (kind == ATTN_SCORE_MOD_ALIBI) {
    sm->alibi_slopes = params;
    return ATTN_OK;
  }
  if (kind == ATTN_SCORE_MOD_REL_BIAS) {
    if (arg < 0 || arg > (1 << 20)) return ATTN_ERR_INVALID_ARG;
    sm->rel_table = params;
    sm->rel_max = arg;
    return ATTN_OK;
  }
  return ATTN_ERR_INVALID_ARG;
}

static attn_status_t validate_dense(const void* q, const void* k, const void* v, const void* o,
                                    const float* lse, int B, int Hq, int Hkv, int Lq, int Lk,
                                    int d, float scale, int mask_kind, int window_l, int window_r,
                                    int draft_block, const int32_t* doc_ids) {
  if (!q || !k || !v || !o || !lse) return ATTN_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(o, 16) ||
      !aligned(lse, 4))
    return ATTN_ERR_INVALID_ARG;
  if (B < 1 || Hq < 1 || Hkv < 1 || Lq < 1 || Lk < 1 || Hq % Hkv != 0) return ATTN_ERR_INVALID_ARG;
  if (!(scale > 0.0f) || !std::isfinite(scale)) return ATTN_ERR_INVALID_ARG;
  if (mask_kind < ATTN_MASK_NONE || mask_kind > ATTN_MASK_DRAFT_BLOCK) return ATTN_ERR_INVALID_ARG;
  if (window_l < -1 || window_r < -1) return ATTN_ERR_INVALID_ARG;
  if (mask_kind == ATTN_MASK_DRAFT_BLOCK && draft_block < 1) return ATTN_ERR_INVALID_ARG;
  if (doc_ids && (!aligned(doc_ids, 4) || Lq > Lk)) return ATTN_ERR_INVALID_ARG;
  if (d != 64 && d != 128) return ATTN_ERR_UNSUPPORTED;
  if (ceil_div(Lk, kBlockN) > attn::kMaxKvTiles) return ATTN_ERR_UNSUPPORTED;
  if ((long long)B * Hq > kMaxGridY) return ATTN_ERR_UNSUPPORTED;
  const long long q_tiles = ceil_div(Lq, kBlockM);
  if ((long long)B * Hq * ((q_tiles + 1) / 2) > 0x7fffffffLL) return ATTN_ERR_UNSUPPORTED;
  return ATTN_OK;
}

// allow_short = false keeps every shape on the persistent kernel (the chunks
// of attn_fwd_host then compute exactly what one attn_fwd call would).
static attn_status_t fwd_dense(const void* q, const void* k, const void* v, void* o, float* lse,
                               int B, int Hq, int Hkv, int Lq, int Lk, int d, float scale,
                               int mask_kind, int window_l, int window_r, int draft_block,
                               const int32_t* doc_ids, const ScoreMod& sm, void* stream,
                               bool allow_short = true) {
  const attn_status_t vs = validate_dense(q, k, v, o, lse, B, Hq, Hkv, Lq, Lk, d, scale,
                                          mask_kind, window_l, window_r, draft_block, doc_ids);
  if (vs != ATTN_OK) return vs;

  FwdParams p;
  std::memset(&p, 0, sizeof p);
  p.o = o;
  p.lse = lse;
  p.doc_ids = doc_ids;
  p.alibi_slopes = sm.alibi_slopes;
  p.rel_table = sm.rel_table;
  p.rel_max = sm.rel_max;
  p.B = B;
  p.Hq = Hq;
  p.Hkv = Hkv;
  p.Lq = Lq;
  p.Lk = Lk;
  p.group = Hq / Hkv;
  p.mask_kind = mask_kind;
  p.window_l = window_l;
  p.window_r = window_r;
  p.draft_block = mask_kind == ATTN_MASK_DRAFT_BLOCK ? draft_block : 1;
  p.scale_log2 = (float)((double)scale * 1.4426950408889634074);
  p.q_tiles = (int)ceil_div(Lq, kBlockM);
  const long long n_units = (long long)B * Hq * ((p.q_tiles + 1) / 2);
  p.n_units = (int)n_units;
  p.err = error_word_for_current_device();
  if (!p.err) return ATTN_ERR_CUDA;

  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  CUtensorMap tq, tk, tv;
  const uint64_t dk[3] = {(uint64_t)d, (uint64_t)Lk, (uint64_t)B * Hkv};
  if (!encode_bf16(&tk, k, 3, dk) || !encode_bf16(&tv, v, 3, dk)) return ATTN_ERR_CUDA;

  // Short queries: a query tile per (b, kv head) leaves most SMs idle in the
  // persistent kernel, so a cluster per row tile splits the visible keys.
  ShortPlan sp;
  if (allow_short && !sm.alibi_slopes && !sm.rel_table &&
      plan_short(B, Hq, Hkv, Lq, Lk, mask_kind, window_l, window_r, p.draft_block, &sp)) {
    p.row_tiles = sp.row_tiles;
    p.key_lo = sp.key_lo;
    p.chunk = sp.chunk;
    p.nsplit = sp.cluster;
    const uint64_t dq2[2] = {(uint64_t)d, (uint64_t)B * Hq * Lq};
    if (!encode_bf16(&tq, q, 2, dq2)) return ATTN_ERR_CUDA;
    cudaError_t e = d == 64 ? attn::launch_short<64>(tq, tk, tv, p, sp.units, st)
                            : attn::launch_short<128>(tq, tk, tv, p, sp.units, st);
    return e == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
  }

  const uint64_t dq[3] = {(uint64_t)d, (uint64_t)Lq, (uint64_t)B * Hq};
  if (!encode_bf16(&tq, q, 3, dq)) return ATTN_ERR_CUDA;
  const int grid = (int)(n_units < num_sms() ? n_units : num_sms());
  cudaError_t e = d == 64 ? attn::launch_prefill<64>(tq, tk, tv, p, grid, st)
                          : attn::launch_prefill<128>(tq, tk, tv, p, grid, st);
  return e == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

attn_status_t attn_fwd(const void* q, const void* k, const void* v, void* o, float* lse, int B,
                       int Hq, int Hkv, int Lq, int Lk, int d, float scale, int mask_kind,
                       int window_l, int window_r, int draft_block, const int32_t* doc_ids,
                       void* stream) {
  return fwd_dense(q, k, v, o, lse, B, Hq, Hkv, Lq, Lk, d, scale, mask_kind, window_l, window_r,
                   draft_block, doc_ids, ScoreMod{}, stream);
}

attn_status_t attn_fwd_score_mod(const void* q, const void* k, const void* v, void* o,
                                 float* lse, int B, int Hq, int Hkv, int Lq, int Lk, int d,
                                 float scale, int mask_kind, int window_l, int window_r,
                                 int draft_block, const int32_t* doc_ids, int score_mod,
                                 const float* score_mod_params, int score_mod_arg, void* stream) {
  ScoreMod sm;
  const attn_status_t st = parse_score_mod(score_mod, score_mod_params, score_mod_arg, &sm);
  if (st != ATTN_OK) return st;
  return fwd_dense(q, k, v, o, lse, B, Hq, Hkv, Lq, Lk, d, scale, mask_kind, window_l, window_r,
                   draft_block, doc_ids, sm, stream);
}

// ------------------------------------------------- host buffers, pipelined
// attn_fwd_host: the inputs and outputs live in host memory.  The work is cut
// into chunks of whole (b, kv head) pairs (with their query heads); chunk c's
// Q, K and V go up on one copy stream while the kernel of chunk c - 1 runs on
// the caller's stream and the O / LSE of chunk c - 2 come down on another, so
// the PCIe transfers in both directions and the kernels overlap.
namespace {

constexpr int kHostChunks = 8;  // target chunk count (fewer when B * Hkv is smaller)

struct HostPipe {
  cudaStream_t h2d = nullptr, d2h = nullptr;
  cudaEvent_t start = nullptr, done = nullptr;
  cudaEvent_t in[kHostChunks] = {}, out[kHostChunks] = {};
};
HostPipe g_pipe[attn::kMaxDevices];
attn::PerContextOnce g_pipe_once;
std::mutex g_pipe_enqueue;  // the events are reused: one enqueue at a time

struct HostLayout {
  size_t q, k, v, o, lse, doc, total;
};

HostLayout host_layout(int B, int Hq, int Hkv, int Lq, int Lk, int d, bool with_doc) {
  auto up = [](size_t x) { return (x + 255) / 256 * 256; };
  HostLayout l;
  const size_t qb = (size_t)B * Hq * Lq * d * 2, kb = (size_t)B * Hkv * Lk * d * 2;
  l.q = 0;
  l.k = up(qb);
  l.v = l.k + up(kb);
  l.o = l.v + up(kb);
  l.lse = l.o + up(qb);
  l.doc = l.lse + up((size_t)B * Hq * Lq * 4);
  l.total = l.doc + (with_doc ? up((size_t)B * Lk * 4) : 0);
  return l;
}

// A chunk: batch elements [b0, b0 + nb) times kv heads [h0, h0 + nh).
struct HostChunk {
  int b0, nb, h0, nh;
};

int plan_host_chunks(int B, int Hkv, HostChunk* out) {
  int n = 0;
  if (B >= kHostChunks) {
    const int nb = (B + kHostChunks - 1) / kHostChunks;
    for (int b0 = 0; b0 < B; b0 += nb) out[n++] = {b0, std::min(nb, B - b0), 0, Hkv};
  } else {
    const int parts = std::min(Hkv, kHostChunks / B);
    const int nh = (Hkv + parts - 1) / parts;
    for (int b = 0; b < B; ++b)
      for (int h0 = 0; h0 < Hkv; h0 += nh) out[n++] = {b, 1, h0, std::min(nh, Hkv - h0)};
  }
  return n;
}

}  // namespace

size_t attn_fwd_host_workspace_size(int B, int Hq, int Hkv, int Lq, int Lk, int d,
                                    int with_doc_ids) {
  if (B < 1 || Hq < 1 || Hkv < 1 || Lq < 1 || Lk < 1 || d < 1 || Hq % Hkv != 0) return 0;
  return host_layout(B, Hq, Hkv, Lq, Lk, d, with_doc_ids != 0).total;
}

attn_status_t attn_fwd_host(const void* q, const void* k, const void* v, void* o, float* lse,
                            int B, int Hq, int Hkv, int Lq, int Lk, int d, float scale,
                            int mask_kind, int window_l, int window_r, int draft_block,
                            const int32_t* doc_ids, void* workspace, size_t ws_bytes,
                            void* stream) {
  if (!q || !k || !v || !o || !lse) return ATTN_ERR_INVALID_ARG;
  if (B < 1 || Hq < 1 || Hkv < 1 || Lq < 1 || Lk < 1 || d < 1 || Hq % Hkv != 0)
    return ATTN_ERR_INVALID_ARG;
  const HostLayout lay = host_layout(B, Hq, Hkv, Lq, Lk, d, doc_ids != nullptr);
  if (!workspace || !aligned(workspace, 256) || ws_bytes < lay.total) return ATTN_ERR_WORKSPACE;
  uint8_t* ws = reinterpret_cast<uint8_t*>(workspace);
  uint8_t *qd = ws + lay.q, *kd = ws + lay.k, *vd = ws + lay.v, *od = ws + lay.o;
  float* ld = reinterpret_cast<float*>(ws + lay.lse);
  int32_t* dd = doc_ids ? reinterpret_cast<int32_t*>(ws + lay.doc) : nullptr;
  // the whole call's arguments, checked on the device-side copies before any work is queued
  const attn_status_t vs = validate_dense(qd, kd, vd, od, ld, B, Hq, Hkv, Lq, Lk, d, scale,
                                          mask_kind, window_l, window_r, draft_block, dd);
  if (vs != ATTN_OK) return vs;
  // chunks stay on the kernel one call over the whole shape would use, so the
  // results match attn_fwd exactly; short-query shapes run as one chunk
  const bool whole_short =
      plan_short_possible(B, Hq, Hkv, Lq, Lk, mask_kind, window_l, window_r, draft_block);
  HostChunk chunks[kHostChunks * 2];
  const int n_chunks = whole_short ? 1 : plan_host_chunks(B, Hkv, chunks);
  if (whole_short) chunks[0] = {0, B, 0, Hkv};

  const cudaError_t se = attn::once_per_context(g_pipe_once, [](int dev) {
    HostPipe& hp = g_pipe[dev];
    cudaError_t e = cudaStreamCreateWithFlags(&hp.h2d, cudaStreamNonBlocking);
    if (e == cudaSuccess) e = cudaStreamCreateWithFlags(&hp.d2h, cudaStreamNonBlocking);
    if (e == cudaSuccess) e = cudaEventCreateWithFlags(&hp.start, cudaEventDisableTiming);
    if (e == cudaSuccess) e = cudaEventCreateWithFlags(&hp.done, cudaEventDisableTiming);
    for (int i = 0; i < kHostChunks && e == cudaSuccess; ++i) {
      e = cudaEventCreateWithFlags(&hp.in[i], cudaEventDisableTiming);
      if (e == cudaSuccess) e = cudaEventCreateWithFlags(&hp.out[i], cudaEventDisableTiming);
    }
    return e;
  });
  if (se != cudaSuccess) return ATTN_ERR_CUDA;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return ATTN_ERR_CUDA;
  HostPipe& hp = g_pipe[dev];
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const int group = Hq / Hkv;
  const size_t qrow = (size_t)Lq * d * 2, krow = (size_t)Lk * d * 2;  // bytes per head

  std::lock_guard<std::mutex> lock(g_pipe_enqueue);
  bool ok = cudaEventRecord(hp.start, st) == cudaSuccess &&
            cudaStreamWaitEvent(hp.h2d, hp.start, 0) == cudaSuccess &&
            cudaStreamWaitEvent(hp.d2h, hp.start, 0) == cudaSuccess;
  if (ok && doc_ids)
    ok = cudaMemcpyAsync(dd, doc_ids, (size_t)B * Lk * 4, cudaMemcpyHostToDevice, hp.h2d) ==
         cudaSuccess;
  for (int c = 0; c < n_chunks && ok; ++c) {
    const HostChunk& ch = chunks[c];
    const size_t qh0 = (size_t)ch.b0 * Hq + (size_t)ch.h0 * group;   // first query head
    const size_t kh0 = (size_t)ch.b0 * Hkv + (size_t)ch.h0;          // first kv head
    const size_t nq = (size_t)ch.nb * ch.nh * group, nk = (size_t)ch.nb * ch.nh;
    ok = cudaMemcpyAsync(qd + qh0 * qrow, static_cast<const uint8_t*>(q) + qh0 * qrow, nq * qrow,
                         cudaMemcpyHostToDevice, hp.h2d) == cudaSuccess &&
         cudaMemcpyAsync(kd + kh0 * krow, static_cast<const uint8_t*>(k) + kh0 * krow, nk * krow,
                         cudaMemcpyHostToDevice, hp.h2d) == cudaSuccess &&
         cudaMemcpyAsync(vd + kh0 * krow, static_cast<const uint8_t*>(v) + kh0 * krow, nk * krow,
                         cudaMemcpyHostToDevice, hp.h2d) == cudaSuccess &&
         cudaEventRecord(hp.in[c], hp.h2d) == cudaSuccess;
  }
  attn_status_t status = ok ? ATTN_OK : ATTN_ERR_CUDA;
  for (int c = 0; c < n_chunks && status == ATTN_OK; ++c) {
    const HostChunk& ch = chunks[c];
    const size_t qh0 = (size_t)ch.b0 * Hq + (size_t)ch.h0 * group;
    const size_t kh0 = (size_t)ch.b0 * Hkv + (size_t)ch.h0;
    const size_t nq = (size_t)ch.nb * ch.nh * group;
    if (cudaStreamWaitEvent(st, hp.in[c], 0) != cudaSuccess) {
      status = ATTN_ERR_CUDA;
      break;
    }
    status = fwd_dense(qd + qh0 * qrow, kd + kh0 * krow, vd + kh0 * krow, od + qh0 * qrow,
                       ld + qh0 * Lq, ch.nb, ch.nh * group, ch.nh, Lq, Lk, d, scale, mask_kind,
                       window_l, window_r, draft_block, dd ? dd + (size_t)ch.b0 * Lk : nullptr,
                       ScoreMod{}, stream, whole_short);
    if (status != ATTN_OK) break;
    if (cudaEventRecord(hp.out[c], st) != cudaSuccess ||
        cudaStreamWaitEvent(hp.d2h, hp.out[c], 0) != cudaSuccess ||
        cudaMemcpyAsync(static_cast<uint8_t*>(o) + qh0 * qrow, od + qh0 * qrow, nq * qrow,
                        cudaMemcpyDeviceToHost, hp.d2h) != cudaSuccess ||
        cudaMemcpyAsync(lse + qh0 * Lq, ld + qh0 * Lq, nq * Lq * 4, cudaMemcpyDeviceToHost,
                        hp.d2h) != cudaSuccess)
      status = ATTN_ERR_CUDA;
  }
  // the caller's stream resumes after the last download, whatever happened above
  if (cudaEventRecord(hp.done, hp.d2h) != cudaSuccess ||
      cudaStreamWaitEvent(st, hp.done, 0) != cudaSuccess)
    status = ATTN_ERR_CUDA;
  return status;
}

static attn_status_t fwd_varlen(const void* q, const void* k, const void* v, void* o, float* lse,
                                const int32_t* cu_seqlens_q, const int32_t* cu_seqlens_k, int B,
                                int Hq, int Hkv, int total_q, int total_k, int max_seqlen_q, int d,
                                float scale, int mask_kind, int window_l, int window_r,
                                int draft_block, const ScoreMod& sm, void* stream) {
  if (!q || !k || !v || !o || !lse || !cu_seqlens_q || !cu_seqlens_k) return ATTN_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(o, 16) ||
      !aligned(lse, 4) || !aligned(cu_seqlens_q, 4) || !aligned(cu_seqlens_k, 4))
    return ATTN_ERR_INVALID_ARG;
  if (B < 1 || Hq < 1 || Hkv < 1 || Hq % Hkv != 0) return ATTN_ERR_INVALID_ARG;
  if (total_q < 1 || total_k < 1 || max_seqlen_q < 1 || max_seqlen_q > total_q)
    return ATTN_ERR_INVALID_ARG;
  if (!(scale > 0.0f) || !std::isfinite(scale)) return ATTN_ERR_INVALID_ARG;
  if (mask_kind < ATTN_MASK_NONE || mask_kind > ATTN_MASK_DRAFT_BLOCK) return ATTN_ERR_INVALID_ARG;
  if (window_l < -1 || window_r < -1) return ATTN_ERR_INVALID_ARG;
  if (mask_kind == ATTN_MASK_DRAFT_BLOCK && draft_block < 1) return ATTN_ERR_INVALID_ARG;
  if (d != 64 && d != 128) return ATTN_ERR_UNSUPPORTED;

  FwdParams p;
  std::memset(&p, 0, sizeof p);
  p.o = o;
  p.lse = lse;
  p.cu_seqlens_q = cu_seqlens_q;
  p.cu_seqlens_k = cu_seqlens_k;
  p.alibi_slopes = sm.alibi_slopes;
  p.rel_table = sm.rel_table;
  p.rel_max = sm.rel_max;
  p.total_q = total_q;
  p.total_k = total_k;
  p.B = B;
  p.Hq = Hq;
  p.Hkv = Hkv;
  p.Lq = max_seqlen_q;  // sizes the units; each sequence's lengths come from cu_seqlens
  p.Lk = 0;
  p.group = Hq / Hkv;
  p.mask_kind = mask_kind;
  p.window_l = window_l;
  p.window_r = window_r;
  p.draft_block = mask_kind == ATTN_MASK_DRAFT_BLOCK ? draft_block : 1;
  p.scale_log2 = (float)((double)scale * 1.4426950408889634074);
  p.q_tiles = (int)ceil_div(max_seqlen_q, kBlockM);
  const long long n_units = (long long)B * Hq * ((p.q_tiles + 1) / 2);
  if (n_units > 0x7fffffffLL) return ATTN_ERR_UNSUPPORTED;
  p.n_units = (int)n_units;
  p.err = error_word_for_current_device();
  if (!p.err) return ATTN_ERR_CUDA;

  CUtensorMap tq, tk, tv;
  if (!encode_bf16_packed(&tq, q, d, Hq, total_q) || !encode_bf16_packed(&tk, k, d, Hkv, total_k) ||
      !encode_bf16_packed(&tv, v, d, Hkv, total_k))
    return ATTN_ERR_CUDA;

  const int grid = (int)(n_units < num_sms() ? n_units : num_sms());
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e = d == 64 ? attn::launch_prefill<64>(tq, tk, tv, p, grid, st)
                          : attn::launch_prefill<128>(tq, tk, tv, p, grid, st);
  return e == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

attn_status_t attn_fwd_varlen(const void* q, const void* k, const void* v, void* o, float* lse,
                              const int32_t* cu_seqlens_q, const int32_t* cu_seqlens_k, int B,
                              int Hq, int Hkv, int total_q, int total_k, int max_seqlen_q, int d,
                              float scale, int mask_kind, int window_l, int window_r,
                              int draft_block, void* stream) {
  return fwd_varlen(q, k, v, o, lse, cu_seqlens_q, cu_seqlens_k, B, Hq, Hkv, total_q, total_k,
                    max_seqlen_q, d, scale, mask_kind, window_l, window_r, draft_block,
                    ScoreMod{}, stream);
}

attn_status_t attn_fwd_varlen_score_mod(const void* q, const void* k, const void* v, void* o,
                                        float* lse, const int32_t* cu_seqlens_q,
                                        const int32_t* cu_seqlens_k, int B, int Hq, int Hkv,
                                        int total_q, int total_k, int max_seqlen_q, int d,
                                        float scale, int mask_kind, int window_l, int window_r,
                                        int draft_block, int score_mod,
                                        const float* score_mod_params, int score_mod_arg,
                                        void* stream) {
  ScoreMod sm;
  const attn_status_t st = parse_score_mod(score_mod, score_mod_params, score_mod_arg, &sm);
  if (st != ATTN_OK) return st;
  return fwd_varlen(q, k, v, o, lse, cu_seqlens_q, cu_seqlens_k, B, Hq, Hkv, total_q, total_k,
                    max_seqlen_q, d, scale, mask_kind, window_l, window_r, draft_block, sm,
                    stream);
}

size_t attn_bwd_workspace_size(int B, int Hq, int Lq, int d) {
  if (B < 1 || Hq < 1 || Lq < 1 || d < 1) return 0;
  const size_t rows = (size_t)B * (size_t)Hq * (size_t)Lq;
  const size_t acc = (rows * (size_t)d * 4 + 255) / 256 * 256;
  return acc + rows * 4;
}

attn_status_t attn_bwd(const void* q, const void* k, const void* v, const void* o,
                       const float* lse, const void* dout, void* dq, void* dk, void* dv, int B,
                       int Hq, int Hkv, int Lq, int Lk, int d, float scale, int mask_kind,
                       int window_l, int window_r, int draft_block, const int32_t* doc_ids,
                       void* workspace, size_t ws_bytes, void* stream) {
  if (!q || !k || !v || !o || !lse || !dout || !dq || !dk || !dv || !workspace)
    return ATTN_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(o, 16) ||
      !aligned(dout, 16) || !aligned(dq, 16) || !aligned(dk, 16) || !aligned(dv, 16) ||
      !aligned(lse, 4) || !aligned(workspace, 256))
    return ATTN_ERR_INVALID_ARG;
  if (B < 1 || Hq < 1 || Hkv < 1 || Lq < 1 || Lk < 1 || Hq % Hkv != 0) return ATTN_ERR_INVALID_ARG;
  if (!(scale > 0.0f) || !std::isfinite(scale)) return ATTN_ERR_INVALID_ARG;
  if (mask_kind < ATTN_MASK_NONE || mask_kind > ATTN_MASK_DRAFT_BLOCK) return ATTN_ERR_INVALID_ARG;
  if (window_l < -1 || window_r < -1) return ATTN_ERR_INVALID_ARG;
  if (mask_kind == ATTN_MASK_DRAFT_BLOCK && draft_block < 1) return ATTN_ERR_INVALID_ARG;
  if (doc_ids && (!aligned(doc_ids, 4) || Lq > Lk)) return ATTN_ERR_INVALID_ARG;
  if (d != 64 && d != 128) return ATTN_ERR_UNSUPPORTED;
  if (ceil_div(Lk, kBlockN) > kMaxGridY || (long long)B * Hkv > 0x7fffffffLL)
    return ATTN_ERR_UNSUPPORTED;
  const size_t need = attn_bwd_workspace_size(B, Hq, Lq, d);
  if (need == 0 || ws_bytes < need) return ATTN_ERR_WORKSPACE;

  attn::BwdParams p;
  std::memset(&p, 0, sizeof p);
  p.o = o;
  p.lse = lse;
  p.dout = dout;
  p.dq = dq;
  p.dk = dk;
  p.dv = dv;
  const size_t rows = (size_t)B * Hq * Lq;
  p.dq_acc = static_cast<float*>(workspace);
  p.dsum = reinterpret_cast<float*>(static_cast<char*>(workspace) +
                                    (rows * (size_t)d * 4 + 255) / 256 * 256);
  p.doc_ids = doc_ids;
  p.B = B;
  p.Hq = Hq;
  p.Hkv = Hkv;
  p.Lq = Lq;
  p.Lk = Lk;
  p.group = Hq / Hkv;
  p.mask_kind = mask_kind;
  p.window_l = window_l;
  p.window_r = window_r;
  p.draft_block = mask_kind == ATTN_MASK_DRAFT_BLOCK ? draft_block : 1;
  p.scale = scale;
  p.scale_log2 = (float)((double)scale * 1.4426950408889634074);
  p.q_tiles = (int)ceil_div(Lq, kBlockM);
  p.err = error_word_for_current_device();
  if (!p.err) return ATTN_ERR_CUDA;

  CUtensorMap tq, tk, tv, tdo, tdq;
  const uint64_t dq3[3] = {(uint64_t)d, (uint64_t)Lq, (uint64_t)B * Hq};
  const uint64_t dk3[3] = {(uint64_t)d, (uint64_t)Lk, (uint64_t)B * Hkv};
  if (!encode_bf16(&tq, q, 3, dq3) || !encode_bf16(&tk, k, 3, dk3) ||
      !encode_bf16(&tv, v, 3, dk3) || !encode_bf16(&tdo, dout, 3, dq3) ||
      !encode_f32_reduce(&tdq, p.dq_acc, dq3))
    return ATTN_ERR_CUDA;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (cudaMemsetAsync(p.dq_acc, 0, rows * (size_t)d * 4, st) != cudaSuccess) return ATTN_ERR_CUDA;
  cudaError_t e = d == 64 ? attn::launch_backward<64>(tq, tk, tv, tdo, tdq, p, st)
                          : attn::launch_backward<128>(tq, tk, tv, tdo, tdq, p, st);
  return e == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

int attn_decode_num_splits(int B, int Hq, int Hkv, int Lq, int Lk_max, int d, int num_splits,
                           int* chunk_keys) {
  SplitPlan pl;
  if (!plan_splits(B, Hq, Hkv, Lq, Lk_max, d, num_splits, &pl)) return -1;
  if (chunk_keys) *chunk_keys = pl.chunk;
  return pl.nsplit;
}

size_t attn_decode_workspace_size(int B, int Hq, int Hkv, int Lq, int Lk_max, int d,
                                  int num_splits) {
  SplitPlan pl;
  if (!plan_splits(B, Hq, Hkv, Lq, Lk_max, d, num_splits, &pl)) return 0;
  const long long nrows = (long long)B * Hq * Lq;
  return ws_lse_offset(pl, nrows, d) + (size_t)pl.nsplit * (size_t)nrows * 4;
}

}  // extern "C"

namespace {

struct PagedKv {
  const int32_t* block_table = nullptr;
  int page_size = 0;
  int pages_per_seq = 0;
  int num_pages = 0;
};

// Fills the launch parameters of the split-KV decode except outputs, workspace
// and score modifier.
void set_decode_shape(FwdParams* p, const int32_t* kv_lens, int B, int Hq, int Hkv, int Lq,
                      int Lk_max, float scale, const SplitPlan& pl, const PagedKv& pg) {
  p->kv_lens = kv_lens;
  p->B = B;
  p->Hq = Hq;
  p->Hkv = Hkv;
  p->Lq = Lq;
  p->Lk = Lk_max;
  p->group = Hq / Hkv;
  p->mask_kind = ATTN_MASK_NONE;
  p->window_l = -1;
  p->window_r = -1;
  p->draft_block = 1;
  p->scale_log2 = (float)((double)scale * 1.4426950408889634074);
  p->chunk = pl.chunk;
  p->nsplit = pl.nsplit;
  p->row_tiles = pl.row_tiles;
  p->block_table = pg.block_table;
  p->page_size = pg.page_size;
  p->pages_per_seq = pg.pages_per_seq;
  p->num_pages = pg.num_pages;
}

// Tensor maps of a bf16 K/V cache: contiguous [planes, rows, d] or a page pool,
// boxes of at most box_rows rows.
bool encode_kv(CUtensorMap* tk, CUtensorMap* tv, const void* k, const void* v, int d,
               uint64_t rows, uint64_t planes, const PagedKv& pg, int Hkv,
               int box_rows = kBlockN) {
  if (pg.block_table) {
    const uint64_t dk[3] = {(uint64_t)d, (uint64_t)pg.page_size,
                            (uint64_t)pg.num_pages * (uint64_t)Hkv};
    const int box = std::min(pg.page_size, box_rows);
    return encode_bf16(tk, k, 3, dk, box) && encode_bf16(tv, v, 3, dk, box);
  }
  const uint64_t dk[3] = {(uint64_t)d, rows, planes};
  return encode_bf16(tk, k, 3, dk, box_rows) && encode_bf16(tv, v, 3, dk, box_rows);
}

// The partial kernel of the split-KV decode for launch parameters p.
attn_status_t launch_split_decode(const FwdParams& p, const void* q, const void* k_cache,
                                  const void* v_cache, int d, const PagedKv& pg,
                                  cudaStream_t st) {
  CUtensorMap tq, tk, tv;
  const uint64_t dq[2] = {(uint64_t)d, (uint64_t)p.B * p.Hq * p.Lq};
  if (!encode_bf16(&tq, q, 2, dq)) return ATTN_ERR_CUDA;
  if (!encode_kv(&tk, &tv, k_cache, v_cache, d, (uint64_t)p.Lk, (uint64_t)p.B * p.Hkv, pg, p.Hkv))
    return ATTN_ERR_CUDA;
  dim3 grid((unsigned)p.nsplit, (unsigned)(p.B * p.Hkv * p.row_tiles), 1);
  const cudaError_t e = d == 64 ? attn::launch_decode<64>(tq, tk, tv, p, grid, st)
                                : attn::launch_decode<128>(tq, tk, tv, p, grid, st);
  return e == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

// Shared body of the contiguous and paged split-KV decode.
attn_status_t decode_impl(const void* q, const void* k_cache, const void* v_cache, void* o,
                          float* lse, const int32_t* kv_lens, int B, int Hq, int Hkv, int Lq,
                          int Lk_max, int d, float scale, int num_splits, void* workspace,
                          size_t ws_bytes, void* stream, const PagedKv& pg, const ScoreMod& sm) {
  if (!q || !k_cache || !v_cache || !o || !lse || !kv_lens) return ATTN_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(o, 16) ||
      !aligned(lse, 4) || !aligned(kv_lens, 4))
    return ATTN_ERR_INVALID_ARG;
  if (!(scale > 0.0f) || !std::isfinite(scale)) return ATTN_ERR_INVALID_ARG;
  SplitPlan pl;
  if (!plan_splits(B, Hq, Hkv, Lq, Lk_max, d, num_splits, &pl)) return ATTN_ERR_INVALID_ARG;
  if (d != 64 && d != 128) return ATTN_ERR_UNSUPPORTED;
  if (pl.chunk / kBlockN > attn::kMaxKvTiles) return ATTN_ERR_UNSUPPORTED;
  const long long nrows = (long long)B * Hq * Lq;
  if (nrows > 0x7fffffffLL) return ATTN_ERR_UNSUPPORTED;
  if ((long long)B * Hkv * pl.row_tiles > kMaxGridY) return ATTN_ERR_UNSUPPORTED;
  const size_t need = attn_decode_workspace_size(B, Hq, Hkv, Lq, Lk_max, d, num_splits);
  if (!workspace || !aligned(workspace, 256) || ws_bytes < need) return ATTN_ERR_WORKSPACE;

  FwdParams p;
  std::memset(&p, 0, sizeof p);
  p.o = o;
  p.lse = lse;
  p.ws_o = reinterpret_cast<float*>(workspace);
  p.ws_lse = reinterpret_cast<float*>(reinterpret_cast<uint8_t*>(workspace) +
                                      ws_lse_offset(pl, nrows, d));
  set_decode_shape(&p, kv_lens, B, Hq, Hkv, Lq, Lk_max, scale, pl, pg);
  p.alibi_slopes = sm.alibi_slopes;
  p.rel_table = sm.rel_table;
  p.rel_max = sm.rel_max;

  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const attn_status_t ds = launch_split_decode(p, q, k_cache, v_cache, d, pg, st);
  if (ds != ATTN_OK) return ds;
  const cudaError_t e = d == 64 ? attn::launch_combine<64>(p, st) : attn::launch_combine<128>(p, st);
  return e == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

}  // namespace

extern "C" {

attn_status_t attn_decode_splitkv(const void* q, const void* k_cache, const void* v_cache,
                                  void* o, float* lse, const int32_t* kv_lens, int B, int Hq,
                                  int Hkv, int Lq, int Lk_max, int d, float scale, int num_splits,
                                  void* workspace, size_t ws_bytes, void* stream) {
  return decode_impl(q, k_cache, v_cache, o, lse, kv_lens, B, Hq, Hkv, Lq, Lk_max, d, scale,
                     num_splits, workspace, ws_bytes, stream, PagedKv{}, ScoreMod{});
}

attn_status_t attn_decode_splitkv_score_mod(const void* q, const void* k_cache,
                                            const void* v_cache, void* o, float* lse,
                                            const int32_t* kv_lens, int B, int Hq, int Hkv,
                                            int Lq, int Lk_max, int d, float scale,
                                            int num_splits, int score_mod,
                                            const float* score_mod_params, int score_mod_arg,
                                            void* workspace, size_t ws_bytes, void* stream) {
  ScoreMod sm;
  const attn_status_t st = parse_score_mod(score_mod, score_mod_params, score_mod_arg, &sm);
  if (st != ATTN_OK) return st;
  return decode_impl(q, k_cache, v_cache, o, lse, kv_lens, B, Hq, Hkv, Lq, Lk_max, d, scale,
                     num_splits, workspace, ws_bytes, stream, PagedKv{}, sm);
}

}  // extern "C"

namespace {

// Checks a paged cache's arguments; fills *pg and *lk, the longest a sequence can be.
attn_status_t parse_paged(const int32_t* block_table, int Hkv, int page_size, int pages_per_seq,
                          int num_pages, PagedKv* pg, int* lk) {
  if (!block_table || !aligned(block_table, 4)) return ATTN_ERR_INVALID_ARG;
  if (page_size < 16 || page_size > (1 << 16) || (page_size & (page_size - 1)) != 0)
    return ATTN_ERR_INVALID_ARG;
  if (pages_per_seq < 1 || num_pages < 1 || Hkv < 1) return ATTN_ERR_INVALID_ARG;
  const long long n = (long long)pages_per_seq * page_size;
  if (n > 0x7fffffffLL) return ATTN_ERR_UNSUPPORTED;
  if ((long long)num_pages * Hkv > 0x7fffffffLL) return ATTN_ERR_UNSUPPORTED;
  pg->block_table = block_table;
  pg->page_size = page_size;
  pg->pages_per_seq = pages_per_seq;
  pg->num_pages = num_pages;
  *lk = (int)n;
  return ATTN_OK;
}

attn_status_t paged_impl(const void* q, const void* k_pages, const void* v_pages,
                         const int32_t* block_table, void* o, float* lse, const int32_t* kv_lens,
                         int B, int Hq, int Hkv, int Lq, int page_size, int pages_per_seq,
                         int num_pages, int d, float scale, int num_splits, void* workspace,
                         size_t ws_bytes, void* stream, const ScoreMod& sm) {
  PagedKv pg;
  int lk = 0;
  const attn_status_t st =
      parse_paged(block_table, Hkv, page_size, pages_per_seq, num_pages, &pg, &lk);
  if (st != ATTN_OK) return st;
  return decode_impl(q, k_pages, v_pages, o, lse, kv_lens, B, Hq, Hkv, Lq, lk, d, scale,
                     num_splits, workspace, ws_bytes, stream, pg, sm);
}

}  // namespace

extern "C" {

attn_status_t attn_decode_paged(const void* q, const void* k_pages, const void* v_pages,
                                const int32_t* block_table, void* o, float* lse,
                                const int32_t* kv_lens, int B, int Hq, int Hkv, int Lq,
                                int page_size, int pages_per_seq, int num_pages, int d,
                                float scale, int num_splits, void* workspace, size_t ws_bytes,
                                void* stream) {
  return paged_impl(q, k_pages, v_pages, block_table, o, lse, kv_lens, B, Hq, Hkv, Lq, page_size,
                    pages_per_seq, num_pages, d, scale, num_splits, workspace, ws_bytes, stream,
                    ScoreMod{});
}

attn_status_t attn_decode_paged_score_mod(const void* q, const void* k_pages, const void* v_pages,
                                          const int32_t* block_table, void* o, float* lse,
                                          const int32_t* kv_lens, int B, int Hq, int Hkv, int Lq,
                                          int page_size, int pages_per_seq, int num_pages, int d,
                                          float scale, int num_splits, int score_mod,
                                          const float* score_mod_params, int score_mod_arg,
                                          void* workspace, size_t ws_bytes, void* stream) {
  ScoreMod sm;
  const attn_status_t st = parse_score_mod(score_mod, score_mod_params, score_mod_arg, &sm);
  if (st != ATTN_OK) return st;
  return paged_impl(q, k_pages, v_pages, block_table, o, lse, kv_lens, B, Hq, Hkv, Lq, page_size,
                    pages_per_seq, num_pages, d, scale, num_splits, workspace, ws_bytes, stream,
                    sm);
}

}  // extern "C"

// ------------------------------------------- decodes with shared-out work
namespace {

int log2_of(int pow2) {
  int s = 0;
  while ((1 << s) < pow2) ++s;
  return s;
}

// CTAs among which a decode's key tiles are shared out (one per SM unless the caller
// asks for a number), and its workspace: two partial results per CTA.
constexpr int kMaxDecodeCtas = 4096;

struct SharePlan {
  int num_ctas, tile_rows, row_tiles, piece;
  size_t part_rows;       // rows of partial results
  size_t lse_off, bytes;  // workspace: O, then the LSEs
};

bool plan_share(int Hq, int Hkv, int Lq, int d, bool q8, int num_ctas, SharePlan* pl) {
  if (Hq < 1 || Hkv < 1 || Lq < 1 || d < 1 || Hq % Hkv) return false;
  if (num_ctas < 0 || num_ctas > kMaxDecodeCtas) return false;
  const long long rows = (long long)(Hq / Hkv) * Lq;
  pl->num_ctas = num_ctas > 0 ? num_ctas : num_sms();
  pl->tile_rows = attn::decode_tile_rows(d, rows);
  pl->piece = attn::piece_tiles(d, q8, pl->tile_rows);
  const long long tiles = ceil_div(rows, pl->tile_rows);
  if (tiles * Hkv > 0x7fffffffLL) return false;
  pl->row_tiles = (int)tiles;
  pl->part_rows = 2 * (size_t)pl->num_ctas * (size_t)pl->tile_rows;
  pl->lse_off = (pl->part_rows * (size_t)d * 4 + 255) / 256 * 256;
  pl->bytes = pl->lse_off + pl->part_rows * 4;
  return true;
}

// Launch parameters of such a decode except its outputs, workspace and scale bytes;
// false for sizes whose 32-bit counters (output rows, keys, the line of work) overflow.
bool set_share_shape(attn::DecodeParams* p, const void* q, const int32_t* kv_lens, int B, int Hq,
                     int Hkv, int Lq, int Lk_max, float scale, const SharePlan& pl,
                     const PagedKv& pg) {
  if (Lk_max > 0x7fffffff - 4096) return false;
  if ((long long)B * Hq > 0x7fffffffLL / Lq) return false;
  const long long unit_cost = ceil_div(Lk_max, kBlockN) + pl.piece;
  if ((long long)B * Hkv > 0x7fffffffLL / pl.row_tiles ||
      (long long)B * Hkv * pl.row_tiles > 0x7fffffffLL / unit_cost)
    return false;
  std::memset(p, 0, sizeof *p);
  p->q = q;
  p->kv_lens = kv_lens;
  p->block_table = pg.block_table;
  p->B = B;
  p->Hq = Hq;
  p->Hkv = Hkv;
  p->Lq = Lq;
  p->Lk = Lk_max;
  p->group = Hq / Hkv;
  p->scale_log2 = (float)((double)scale * 1.4426950408889634074);
  p->num_ctas = pl.num_ctas;
  p->tile_rows = pl.tile_rows;
  p->piece = pl.piece;
  p->row_tiles = pl.row_tiles;
  p->page_size = pg.page_size;
  p->page_shift = pg.block_table ? log2_of(pg.page_size) : 0;
  p->pages_per_seq = pg.pages_per_seq;
  p->num_pages = pg.num_pages;
  return true;
}

}  // namespace

// ------------------------------------------------------- shared prefix
namespace {

constexpr int kMaxPrefix = 0x7fffffff - (1 << 20);  // key counters are 32-bit

// Splits of the prefix: row tiles (128 rows of one KV head, whatever their
// sequence) in pairs, and np chunks of whole key tiles.
struct PrefixPlan {
  int nb, per_seq, tiles, pairs, box_rows;
  int np, chunk;
  int cache_ctas;  // CTAs for the sequences' own caches
};

// How many CTAs work on the prefix, and how many on the sequences' own caches where
// their decode shares its key tiles out (few query rows).  The two kernels do not
// depend on each other and take one CTA per SM each, so they either run one after the
// other on all SMs or, where the prefix's CTAs leave SMs free, side by side: one
// start-up fewer, and the slower of the two counts.  Costs, in units of one key tile of
// a prefix CTA (1.9 us at d = 128): the prefix rounds of CTAs over the SMs x (tiles per
// CTA + 4), the caches 6 + 0.48 per tile of a CTA's share (d = 64: 0.27) counted as
// decode_sched.cuh does, for full caches; each split's partial rows, written and read
// back, 0.06 + 1.5e-4 per row.  Side by side the prefix may take at most
// 1.4 times its least time, which bounds the loss where the caches hold much
// less.  Measured one after the other / side by side as planned, us: 4 sequences x 8 KV
// heads, 2064 + 129 keys, d = 128: 17.1 / 13.7; 24 x 4 heads, 8190 + 2064 keys,
// d = 64, 16 rows: 35.1 / 28.1; 16 x 8 heads, 2064 + 1000 keys: 28.1 / 21.9; 64 x 8
// heads, 4096 + 256 keys, 8 rows: 45.2 / 39.7.
bool plan_prefix(int B, int Hq, int Hkv, int Lq, int Lp, int Lk_max, int d, int num_splits,
                 PrefixPlan* pp) {
  if (B < 1 || Hq < 1 || Hkv < 1 || Lq < 1 || Lp < 1 || Lk_max < 1 || num_splits < 0 || Hq % Hkv)
    return false;
  if (Lp > kMaxPrefix) return false;
  const long long G = (long long)(Hq / Hkv) * Lq;
  if (G > 0x7fffffffLL / 2) return false;
  pp->nb = G <= kBlockM ? (int)std::min<long long>(kBlockM / G, B) : 1;
  pp->per_seq = (int)ceil_div(G, kBlockM);
  const long long tiles = G <= kBlockM ? ceil_div(B, pp->nb) : (long long)B * pp->per_seq;
  if (tiles > 0x7fffffffLL) return false;
  pp->tiles = (int)tiles;
  pp->pairs = (int)ceil_div(tiles, 2);
  pp->box_rows = G <= kBlockM ? (int)G * pp->nb : kBlockM;
  const long long key_tiles = ceil_div(Lp, kBlockN), sms = num_sms();
  const long long units = (long long)Hkv * pp->pairs;
  if (units > 0x7fffffffLL) return false;
  const bool shares = attn::decode_tile_rows(d, G) < kBlockM;
  const double cache_work = (double)B * Hkv *
                            ((double)ceil_div(Lk_max, kBlockN) +
                             attn::piece_tiles(d, false, attn::decode_tile_rows(d, G))) *
                            (d == 64 ? 0.27 : 0.48);
  const double partials = 0.06 + (double)B * Hq * Lq * 1.5e-4;
  struct Choice {
    long long tiles, np, ctas;  // key tiles per split, splits, CTAs of the prefix
    double prefix;              // its time
  };
  auto choice = [&](long long n) {
    Choice c;
    c.tiles = ceil_div(key_tiles, n);
    c.np = ceil_div(key_tiles, c.tiles);
    c.ctas = units * c.np;
    c.prefix = (double)ceil_div(c.ctas, sms) * ((double)c.tiles + 4.0) + (double)c.np * partials;
    return c;
  };
  auto in_turn = [&](const Choice& c) {
    return c.prefix + (shares ? 6.0 + cache_work / (double)sms : 0.0);
  };
  auto abreast = [&](const Choice& c) {  // c.ctas < sms
    const double cache = 6.0 + cache_work / (double)(sms - c.ctas);
    return std::max(c.prefix, cache) + 0.1 * std::min(c.prefix, cache);
  };
  // every count that one round of CTAs holds, and for two to four rounds the largest
  const long long asked = std::min<long long>(num_splits, key_tiles);
  const long long one_round = std::max<long long>(std::min(key_tiles, sms / units), 1);
  Choice best = choice(asked > 0 ? asked : 1);
  if (asked == 0) {
    for (long long n = 2; n <= one_round; ++n) {
      const Choice c = choice(n);
      if (c.prefix < best.prefix) best = c;
    }
    for (long long r = 2; r <= 4; ++r) {
      const Choice c = choice(std::max<long long>(std::min(key_tiles, r * sms / units), 1));
      if (c.prefix < best.prefix) best = c;
    }
  }
  bool side = false;
  if (shares) {
    double cost = in_turn(best);
    const double limit = 1.4 * (best.prefix + 5.0) - 5.0;  // 5: the rest of the call
    for (long long n = asked > 0 ? asked : 1; n <= (asked > 0 ? asked : one_round); ++n) {
      const Choice c = choice(n);
      if (c.ctas >= sms) break;
      const double a = side ? abreast(c) : 1.05 * abreast(c);  // in turn unless clearly better
      if (c.prefix <= limit && a < cost) {
        best = c;
        cost = abreast(c);
        side = true;
      }
    }
  }
  pp->chunk = (int)(best.tiles * kBlockN);
  pp->np = (int)best.np;
  pp->cache_ctas = (int)(side ? sms - best.ctas : sms);
  return true;
}

// The whole call.  The sequences' own caches: with few query rows per KV head the
// decode that shares its key tiles out (share), else the split-KV decode (split).
// Workspace: fp32 partial outputs, the prefix's np splits first, then one row per
// output row and two partial results per CTA (share) or the splits' (split); then, 256-byte
// aligned, their LSEs in the same order.
struct PrefixCall {
  PrefixPlan pp;
  bool few_rows;
  SharePlan share;
  SplitPlan split;
  long long nrows;
  size_t part_rows;  // rows of partial results
  size_t lse_off, bytes;
};

bool plan_prefix_call(int B, int Hq, int Hkv, int Lq, int Lp, int Lk_max, int d, int num_splits,
                      PrefixCall* pc) {
  if (!plan_prefix(B, Hq, Hkv, Lq, Lp, Lk_max, d, num_splits, &pc->pp)) return false;
  if (!plan_share(Hq, Hkv, Lq, d, false, 0, &pc->share)) return false;
  pc->share.num_ctas = pc->pp.cache_ctas;  // the workspace has room for one per SM
  if (!plan_splits(B, Hq, Hkv, Lq, Lk_max, d, 0, &pc->split)) return false;
  if ((long long)B * Hq > 0x7fffffffLL / Lq) return false;
  pc->nrows = (long long)B * Hq * Lq;
  pc->few_rows = pc->share.tile_rows < kBlockM;
  const size_t n = (size_t)pc->nrows;
  pc->part_rows = pc->few_rows ? (pc->pp.np + 1) * n + pc->share.part_rows
                               : ((size_t)pc->pp.np + pc->split.nsplit) * n;
  pc->lse_off = (pc->part_rows * (size_t)d * 4 + 255) / 256 * 256;
  pc->bytes = pc->lse_off + pc->part_rows * 4;
  return true;
}

attn_status_t shared_prefix_impl(const void* q, const void* k_prefix, const void* v_prefix,
                                 const int32_t* prefix_table, const void* k_cache,
                                 const void* v_cache, void* o, float* lse, const int32_t* kv_lens,
                                 int B, int Hq, int Hkv, int Lq, int Lp, int Lk_max, int d,
                                 float scale, int num_splits, void* workspace, size_t ws_bytes,
                                 void* stream, const PagedKv& pg) {
  if (!q || !k_prefix || !v_prefix || !k_cache || !v_cache || !o || !lse || !kv_lens)
    return ATTN_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(k_prefix, 16) || !aligned(v_prefix, 16) ||
      !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(o, 16) || !aligned(lse, 4) ||
      !aligned(kv_lens, 4))
    return ATTN_ERR_INVALID_ARG;
  if (!(scale > 0.0f) || !std::isfinite(scale)) return ATTN_ERR_INVALID_ARG;
  if (B < 1 || Hq < 1 || Hkv < 1 || Lq < 1 || Lp < 1 || Lk_max < 1 || num_splits < 0 || Hq % Hkv)
    return ATTN_ERR_INVALID_ARG;
  if (d != 64 && d != 128) return ATTN_ERR_UNSUPPORTED;
  PrefixCall pc;
  if (!plan_prefix_call(B, Hq, Hkv, Lq, Lp, Lk_max, d, num_splits, &pc))
    return ATTN_ERR_UNSUPPORTED;
  attn::DecodeParams sh;
  if (pc.few_rows) {
    if (!set_share_shape(&sh, q, kv_lens, B, Hq, Hkv, Lq, Lk_max, scale, pc.share, pg))
      return ATTN_ERR_UNSUPPORTED;
  } else {
    if (pc.split.chunk / kBlockN > attn::kMaxKvTiles) return ATTN_ERR_UNSUPPORTED;
    if ((long long)B * Hkv * pc.split.row_tiles > kMaxGridY) return ATTN_ERR_UNSUPPORTED;
  }
  if ((long long)Hkv * pc.pp.pairs * pc.pp.np > 0x7fffffffLL) return ATTN_ERR_UNSUPPORTED;
  if (!workspace || !aligned(workspace, 256) || ws_bytes < pc.bytes) return ATTN_ERR_WORKSPACE;
  int* err = error_word_for_current_device();
  if (!err) return ATTN_ERR_CUDA;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const int np = pc.pp.np, G = Hq / Hkv * Lq;
  const size_t n = (size_t)pc.nrows;
  float* ws_o = reinterpret_cast<float*>(workspace);
  float* ws_lse = reinterpret_cast<float*>(reinterpret_cast<uint8_t*>(workspace) + pc.lse_off);
  attn::PrefixParams x;
  std::memset(&x, 0, sizeof x);
  x.ws_o = ws_o;
  x.ws_lse = ws_lse;
  x.err = err;
  x.prefix_table = prefix_table;
  x.nrows = pc.nrows;
  x.B = B;
  x.Hkv = Hkv;
  x.G = G;
  x.Lp = Lp;
  x.nb = pc.pp.nb;
  x.per_seq = pc.pp.per_seq;
  x.tiles = pc.pp.tiles;
  x.pairs = pc.pp.pairs;
  x.box_rows = pc.pp.box_rows;
  x.chunk = pc.pp.chunk;
  x.nsplit = np;
  x.page_size = pg.page_size;
  x.num_pages = pg.num_pages;
  x.scale_log2 = (float)((double)scale * 1.4426950408889634074);
  CUtensorMap tq, tk, tv;
  if (!encode_bf16_rows(&tq, q, d, G, Hkv, B, std::min(G, kBlockM), pc.pp.nb)) return ATTN_ERR_CUDA;
  if (!encode_kv(&tk, &tv, k_prefix, v_prefix, d, (uint64_t)Lp, (uint64_t)Hkv, pg, Hkv))
    return ATTN_ERR_CUDA;
  cudaError_t e = d == 64 ? attn::launch_prefix<64>(tq, tk, tv, x, st)
                          : attn::launch_prefix<128>(tq, tk, tv, x, st);
  if (e != cudaSuccess) return ATTN_ERR_CUDA;

  if (pc.few_rows) {
    sh.o = o;
    sh.lse = lse;
    sh.prefix_o = ws_o;
    sh.prefix_lse = ws_lse;
    sh.num_prefix = np;
    sh.own_o = ws_o + np * n * d;
    sh.own_lse = ws_lse + np * n;
    sh.ws_o = sh.own_o + n * d;
    sh.ws_lse = sh.own_lse + n;
    sh.err = err;
    CUtensorMap ck, cv;
    if (!encode_kv(&ck, &cv, k_cache, v_cache, d, (uint64_t)Lk_max, (uint64_t)B * Hkv, pg, Hkv,
                   attn::decode_rows_box(d, false, kBlockN)))
      return ATTN_ERR_CUDA;
    e = d == 64 ? attn::launch_decode_rows<64, false>(ck, cv, sh, st)
                : attn::launch_decode_rows<128, false>(ck, cv, sh, st);
    if (e != cudaSuccess) return ATTN_ERR_CUDA;
    e = d == 64 ? attn::launch_decode_merge<64>(sh, num_sms(), st)
                : attn::launch_decode_merge<128>(sh, num_sms(), st);
    return e == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
  }

  // partials: splits [0, np) the prefix, [np, np + nsplit) the sequences' own caches
  FwdParams p;
  std::memset(&p, 0, sizeof p);
  set_decode_shape(&p, kv_lens, B, Hq, Hkv, Lq, Lk_max, scale, pc.split, pg);
  p.ws_o = ws_o + np * n * d;
  p.ws_lse = ws_lse + np * n;
  const attn_status_t ds = launch_split_decode(p, q, k_cache, v_cache, d, pg, st);
  if (ds != ATTN_OK) return ds;
  p.o = o;
  p.lse = lse;
  p.ws_o = ws_o;
  p.ws_lse = ws_lse;
  p.nsplit = np + pc.split.nsplit;
  e = d == 64 ? attn::launch_combine<64>(p, st) : attn::launch_combine<128>(p, st);
  return e == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

}  // namespace

extern "C" {

int attn_decode_shared_prefix_num_splits(int B, int Hq, int Hkv, int Lq, int Lp, int Lk_max, int d,
                                         int num_splits, int* chunk_keys) {
  PrefixPlan pp;
  if (!plan_prefix(B, Hq, Hkv, Lq, Lp, Lk_max, d, num_splits, &pp)) return -1;
  if (chunk_keys) *chunk_keys = pp.chunk;
  return pp.np;
}

size_t attn_decode_shared_prefix_workspace_size(int B, int Hq, int Hkv, int Lq, int Lp, int Lk_max,
                                                int d, int num_splits) {
  PrefixCall pc;
  if (!plan_prefix_call(B, Hq, Hkv, Lq, Lp, Lk_max, d, num_splits, &pc)) return 0;
  return pc.bytes;
}

attn_status_t attn_decode_shared_prefix(const void* q, const void* k_prefix, const void* v_prefix,
                                        const void* k_cache, const void* v_cache, void* o,
                                        float* lse, const int32_t* kv_lens, int B, int Hq, int Hkv,
                                        int Lq, int Lp, int Lk_max, int d, float scale,
                                        int num_splits, void* workspace, size_t ws_bytes,
                                        void* stream) {
  return shared_prefix_impl(q, k_prefix, v_prefix, nullptr, k_cache, v_cache, o, lse, kv_lens, B,
                            Hq, Hkv, Lq, Lp, Lk_max, d, scale, num_splits, workspace, ws_bytes,
                            stream, PagedKv{});
}

attn_status_t attn_decode_shared_prefix_paged(
    const void* q, const void* k_pages, const void* v_pages, const int32_t* prefix_table,
    const int32_t* block_table, void* o, float* lse, const int32_t* kv_lens, int B, int Hq,
    int Hkv, int Lq, int Lp, int page_size, int pages_per_seq, int num_pages, int d, float scale,
    int num_splits, void* workspace, size_t ws_bytes, void* stream) {
  PagedKv pg;
  int lk = 0;
  if (!prefix_table || !aligned(prefix_table, 4)) return ATTN_ERR_INVALID_ARG;
  const attn_status_t st =
      parse_paged(block_table, Hkv, page_size, pages_per_seq, num_pages, &pg, &lk);
  if (st != ATTN_OK) return st;
  return shared_prefix_impl(q, k_pages, v_pages, prefix_table, k_pages, v_pages, o, lse, kv_lens,
                            B, Hq, Hkv, Lq, Lp, lk, d, scale, num_splits, workspace, ws_bytes,
                            stream, pg);
}

}  // extern "C"

// ------------------------------------------------------- 8-bit KV cache
namespace {

// Rows of one call: row counters are 32-bit, with room for the last block's, and so is
// the number of a block's (sequence, head) pair, which the grid rounds up to a multiple of
// 65535.
constexpr long long kMaxCacheRows = 0x7fffffffLL - 65535;

// Arguments shared by append and read-back.
attn_status_t cache_params(const void* k_codes, const void* v_codes, const uint8_t* k_exp,
                           const uint8_t* v_exp, const int32_t* kv_lens, int B, int Hkv, int Lk,
                           int d, const PagedKv& pg, attn::CacheParams* p) {
  if (!k_codes || !v_codes || !k_exp || !v_exp || !kv_lens) return ATTN_ERR_INVALID_ARG;
  if (!aligned(k_codes, 16) || !aligned(v_codes, 16) || !aligned(kv_lens, 4))
    return ATTN_ERR_INVALID_ARG;
  if (B < 1 || Hkv < 1 || Lk < 1) return ATTN_ERR_INVALID_ARG;
  if (d != 64 && d != 128) return ATTN_ERR_UNSUPPORTED;
  std::memset(p, 0, sizeof *p);
  p->k_codes = const_cast<void*>(k_codes);
  p->v_codes = const_cast<void*>(v_codes);
  p->k_exp = const_cast<uint8_t*>(k_exp);
  p->v_exp = const_cast<uint8_t*>(v_exp);
  p->kv_lens = kv_lens;
  p->B = B;
  p->Hkv = Hkv;
  p->Lk = Lk;
  p->block_table = pg.block_table;
  p->page_shift = pg.block_table ? log2_of(pg.page_size) : 0;
  p->pages_per_seq = pg.pages_per_seq;
  p->num_pages = pg.num_pages;
  return ATTN_OK;
}

attn_status_t append_impl(const void* k, const void* v, void* k_codes, void* v_codes,
                          uint8_t* k_exp, uint8_t* v_exp, const int32_t* kv_lens,
                          const int32_t* new_lens, int B, int Hkv, int Ln, int Lk, int d,
                          const PagedKv& pg, void* stream) {
  attn::CacheParams p;
  const attn_status_t vs =
      cache_params(k_codes, v_codes, k_exp, v_exp, kv_lens, B, Hkv, Lk, d, pg, &p);
  if (vs != ATTN_OK) return vs;
  if (!k || !v || !aligned(k, 16) || !aligned(v, 16)) return ATTN_ERR_INVALID_ARG;
  if (Ln < 1 || (new_lens && !aligned(new_lens, 4))) return ATTN_ERR_INVALID_ARG;
  if ((long long)B * Hkv > kMaxCacheRows / Ln) return ATTN_ERR_UNSUPPORTED;
  p.k_in = k;
  p.v_in = v;
  p.new_lens = new_lens;
  p.Ln = Ln;
  p.err = error_word_for_current_device();
  if (!p.err) return ATTN_ERR_CUDA;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e =
      d == 64 ? attn::launch_cache_append<64>(p, num_sms(), st)
              : attn::launch_cache_append<128>(p, num_sms(), st);
  return e == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

attn_status_t read_impl(const void* k_codes, const void* v_codes, const uint8_t* k_exp,
                        const uint8_t* v_exp, const int32_t* kv_lens, void* k, void* v, int B,
                        int Hkv, int Lk, int d, const PagedKv& pg, void* stream) {
  attn::CacheParams p;
  const attn_status_t vs =
      cache_params(k_codes, v_codes, k_exp, v_exp, kv_lens, B, Hkv, Lk, d, pg, &p);
  if (vs != ATTN_OK) return vs;
  if (!k || !v || !aligned(k, 16) || !aligned(v, 16)) return ATTN_ERR_INVALID_ARG;
  if ((long long)B * Hkv > kMaxCacheRows / Lk) return ATTN_ERR_UNSUPPORTED;
  p.k_out = k;
  p.v_out = v;
  p.err = error_word_for_current_device();
  if (!p.err) return ATTN_ERR_CUDA;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e =
      d == 64 ? attn::launch_cache_read<64>(p, num_sms(), st)
              : attn::launch_cache_read<128>(p, num_sms(), st);
  return e == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

attn_status_t decode_q8_impl(const void* q, const void* k_codes, const void* v_codes,
                             const uint8_t* k_exp, const uint8_t* v_exp, void* o, float* lse,
                             const int32_t* kv_lens, int B, int Hq, int Hkv, int Lq, int Lk_max,
                             int d, float scale, int num_ctas, void* workspace, size_t ws_bytes,
                             void* stream, const PagedKv& pg) {
  if (!q || !k_codes || !v_codes || !k_exp || !v_exp || !o || !lse || !kv_lens)
    return ATTN_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(k_codes, 16) || !aligned(v_codes, 16) || !aligned(o, 16) ||
      !aligned(lse, 4) || !aligned(kv_lens, 4))
    return ATTN_ERR_INVALID_ARG;
  if (!(scale > 0.0f) || !std::isfinite(scale)) return ATTN_ERR_INVALID_ARG;
  SharePlan pl;
  if (B < 1 || Lk_max < 1 || !plan_share(Hq, Hkv, Lq, d, true, num_ctas, &pl))
    return ATTN_ERR_INVALID_ARG;
  if (d != 64 && d != 128) return ATTN_ERR_UNSUPPORTED;
  attn::DecodeParams p;
  if (!set_share_shape(&p, q, kv_lens, B, Hq, Hkv, Lq, Lk_max, scale, pl, pg))
    return ATTN_ERR_UNSUPPORTED;
  if (!workspace || !aligned(workspace, 256) || ws_bytes < pl.bytes) return ATTN_ERR_WORKSPACE;
  p.o = o;
  p.lse = lse;
  p.ws_o = reinterpret_cast<float*>(workspace);
  p.ws_lse = reinterpret_cast<float*>(reinterpret_cast<uint8_t*>(workspace) + pl.lse_off);
  p.k_codes = k_codes;
  p.v_codes = v_codes;
  p.k_exp = k_exp;
  p.v_exp = v_exp;
  p.err = error_word_for_current_device();
  if (!p.err) return ATTN_ERR_CUDA;

  CUtensorMap tk, tv;
  const uint64_t rows = pg.block_table ? (uint64_t)pg.page_size : (uint64_t)Lk_max;
  const uint64_t planes =
      pg.block_table ? (uint64_t)pg.num_pages * (uint64_t)Hkv : (uint64_t)B * (uint64_t)Hkv;
  const uint64_t dims[3] = {(uint64_t)d, rows, planes};
  const bool wide = pl.tile_rows == kBlockM;
  const int page_rows = pg.block_table ? pg.page_size : 1 << 16;
  const int box = wide ? std::min(page_rows, 64) : attn::decode_rows_box(d, true, page_rows);
  if (!encode_codes(&tk, k_codes, dims, box) || !encode_codes(&tv, v_codes, dims, box))
    return ATTN_ERR_CUDA;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (wide) {
    CUtensorMap tq;
    const uint64_t dq[2] = {(uint64_t)d, (uint64_t)B * Hq * Lq};
    if (!encode_bf16(&tq, q, 2, dq)) return ATTN_ERR_CUDA;
    e = d == 64 ? attn::launch_decode_q8_wide<64>(tq, tk, tv, p, st)
                : attn::launch_decode_q8_wide<128>(tq, tk, tv, p, st);
  } else {
    e = d == 64 ? attn::launch_decode_rows<64, true>(tk, tv, p, st)
                : attn::launch_decode_rows<128, true>(tk, tv, p, st);
  }
  if (e != cudaSuccess) return ATTN_ERR_CUDA;
  e = d == 64 ? attn::launch_decode_merge<64>(p, num_sms(), st)
              : attn::launch_decode_merge<128>(p, num_sms(), st);
  return e == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

}  // namespace

extern "C" {

attn_status_t attn_cache_append_q8(const void* k, const void* v, void* k_cache, void* v_cache,
                                   uint8_t* k_exp, uint8_t* v_exp, const int32_t* kv_lens,
                                   const int32_t* new_lens, int B, int Hkv, int Ln, int Lk_max,
                                   int d, void* stream) {
  return append_impl(k, v, k_cache, v_cache, k_exp, v_exp, kv_lens, new_lens, B, Hkv, Ln, Lk_max,
                     d, PagedKv{}, stream);
}

attn_status_t attn_cache_append_paged_q8(const void* k, const void* v, void* k_pages,
                                         void* v_pages, uint8_t* k_exp, uint8_t* v_exp,
                                         const int32_t* block_table, const int32_t* kv_lens,
                                         const int32_t* new_lens, int B, int Hkv, int Ln,
                                         int page_size, int pages_per_seq, int num_pages, int d,
                                         void* stream) {
  PagedKv pg;
  int lk = 0;
  const attn_status_t st =
      parse_paged(block_table, Hkv, page_size, pages_per_seq, num_pages, &pg, &lk);
  if (st != ATTN_OK) return st;
  return append_impl(k, v, k_pages, v_pages, k_exp, v_exp, kv_lens, new_lens, B, Hkv, Ln, lk, d,
                     pg, stream);
}

attn_status_t attn_cache_read_q8(const void* k_cache, const void* v_cache, const uint8_t* k_exp,
                                 const uint8_t* v_exp, const int32_t* kv_lens, void* k, void* v,
                                 int B, int Hkv, int Lk_max, int d, void* stream) {
  return read_impl(k_cache, v_cache, k_exp, v_exp, kv_lens, k, v, B, Hkv, Lk_max, d, PagedKv{},
                   stream);
}

attn_status_t attn_cache_read_paged_q8(const void* k_pages, const void* v_pages,
                                       const uint8_t* k_exp, const uint8_t* v_exp,
                                       const int32_t* block_table, const int32_t* kv_lens,
                                       void* k, void* v, int B, int Hkv, int page_size,
                                       int pages_per_seq, int num_pages, int d, void* stream) {
  PagedKv pg;
  int lk = 0;
  const attn_status_t st =
      parse_paged(block_table, Hkv, page_size, pages_per_seq, num_pages, &pg, &lk);
  if (st != ATTN_OK) return st;
  return read_impl(k_pages, v_pages, k_exp, v_exp, kv_lens, k, v, B, Hkv, lk, d, pg, stream);
}

size_t attn_decode_q8_workspace_size(int Hq, int Hkv, int Lq, int d, int num_ctas) {
  SharePlan pl;
  return plan_share(Hq, Hkv, Lq, d, true, num_ctas, &pl) ? pl.bytes : 0;
}

attn_status_t attn_decode_splitkv_q8(const void* q, const void* k_cache, const void* v_cache,
                                     const uint8_t* k_exp, const uint8_t* v_exp, void* o,
                                     float* lse, const int32_t* kv_lens, int B, int Hq, int Hkv,
                                     int Lq, int Lk_max, int d, float scale, int num_ctas,
                                     void* workspace, size_t ws_bytes, void* stream) {
  return decode_q8_impl(q, k_cache, v_cache, k_exp, v_exp, o, lse, kv_lens, B, Hq, Hkv, Lq,
                        Lk_max, d, scale, num_ctas, workspace, ws_bytes, stream, PagedKv{});
}

attn_status_t attn_decode_paged_q8(const void* q, const void* k_pages, const void* v_pages,
                                   const uint8_t* k_exp, const uint8_t* v_exp,
                                   const int32_t* block_table, void* o, float* lse,
                                   const int32_t* kv_lens, int B, int Hq, int Hkv, int Lq,
                                   int page_size, int pages_per_seq, int num_pages, int d,
                                   float scale, int num_ctas, void* workspace, size_t ws_bytes,
                                   void* stream) {
  PagedKv pg;
  int lk = 0;
  const attn_status_t st =
      parse_paged(block_table, Hkv, page_size, pages_per_seq, num_pages, &pg, &lk);
  if (st != ATTN_OK) return st;
  return decode_q8_impl(q, k_pages, v_pages, k_exp, v_exp, o, lse, kv_lens, B, Hq, Hkv, Lq, lk, d,
                        scale, num_ctas, workspace, ws_bytes, stream, pg);
}

}  // extern "C"

extern "C" {

attn_status_t attn_get_device_error(void* stream, int* raw_bits) {
  if (raw_bits) *raw_bits = 0;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (cudaStreamSynchronize(st) != cudaSuccess) return ATTN_ERR_CUDA;
  int* word = attn::device_error_word();
  if (!word) return ATTN_ERR_CUDA;
  int bits = 0;
  if (cudaMemcpy(&bits, word, sizeof bits, cudaMemcpyDeviceToHost) != cudaSuccess)
    return ATTN_ERR_CUDA;
  const int zero = 0;
  if (cudaMemcpy(word, &zero, sizeof zero, cudaMemcpyHostToDevice) != cudaSuccess)
    return ATTN_ERR_CUDA;
  if (raw_bits) *raw_bits = bits;
  if (bits & (attn::kDevErrTimeoutProducer | attn::kDevErrTimeoutMma |
              attn::kDevErrTimeoutSoftmax | attn::kDevErrTimeoutSelftest))
    return ATTN_ERR_TIMEOUT;
  if (bits & (attn::kDevErrBadKvLen | attn::kDevErrBadPage | attn::kDevErrBadSeqlens))
    return ATTN_ERR_INVALID_ARG;
  return ATTN_OK;
}

attn_status_t attn_selftest_wait_timeout(void* stream) {
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  return attn::launch_selftest_wait(st) == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

}  // extern "C"
