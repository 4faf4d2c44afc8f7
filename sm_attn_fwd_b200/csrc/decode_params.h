// Launch parameters of the 8-bit cache's kernels and of the decodes that share out their
// work (decode_sched.cuh), used by host and device.
#pragma once

#include <cstdint>

namespace attn {

// Writing (append) and reading back an 8-bit cache.  Cache rows: contiguous
// [B, Hkv, Lk] or, with a block table, [num_pages, Hkv, page_size].
struct CacheParams {
  const void* k_in;  // append: bf16 [B, Hkv, Ln, d]
  const void* v_in;
  void* k_out;       // read: bf16 [B, Hkv, Lk, d]
  void* v_out;
  void* k_codes;     // e4m3 codes, d per row
  void* v_codes;
  uint8_t* k_exp;    // scale byte per row
  uint8_t* v_exp;
  const int32_t* kv_lens;      // [B]
  const int32_t* new_lens;     // append: [B] or null (Ln each)
  const int32_t* block_table;  // [B, pages_per_seq] or null
  int* err;
  int B, Hkv, Ln, Lk;  // Lk: longest a sequence can be (pages_per_seq * page_size when paged)
  int page_shift;      // log2(page_size)
  int pages_per_seq, num_pages;
};

// Decode over an 8-bit cache, or a bf16 one with few query rows.  The work is shared among
// num_ctas CTAs as decode_sched.cuh describes; CTA c's partial results are slots 2 c and
// 2 c + 1 of the workspace.
struct DecodeParams {
  const void* q;  // bf16 [B, Hq, Lq, d]
  void* o;        // bf16 [B, Hq, Lq, d]
  float* lse;     // fp32 [B, Hq, Lq]
  float* ws_o;    // fp32 [2 num_ctas, tile_rows, d]
  float* ws_lse;  // fp32 [2 num_ctas, tile_rows]
  // behind a shared prefix: its splits' partial results, and where the units that one
  // CTA computes go instead of o and lse (null otherwise)
  const float* prefix_o;    // fp32 [num_prefix, B*Hq*Lq, d]
  const float* prefix_lse;  // fp32 [num_prefix, B*Hq*Lq]
  float* own_o;             // fp32 [B*Hq*Lq, d]
  float* own_lse;           // fp32 [B*Hq*Lq]
  int num_prefix;
  const void* k_codes;  // 8-bit cache: codes and scale bytes
  const void* v_codes;
  const uint8_t* k_exp;
  const uint8_t* v_exp;
  const int32_t* kv_lens;
  const int32_t* block_table;
  int* err;
  int B, Hq, Hkv, Lq, Lk, group;
  float scale_log2;
  int num_ctas;
  int tile_rows;  // query rows of a unit: 8, 16, 32 or 128
  int row_tiles;  // units per (b, kv head): ceil(group * Lq / tile_rows)
  int piece;      // piece_tiles()
  int page_size, page_shift, pages_per_seq, num_pages;
};

// Cost, in key tiles, of starting on and finishing a unit (decode_sched.cuh).  A tile of
// an 8-bit cache at d = 64 is half the bytes of any other, so it counts more of them:
// 16 x 16 heads, 1 to 4099 keys, one row: 27.6 us with 5, 29.7 with 3.  Elsewhere the two lie
// within 5 % of each other, on either side.  With 3 and with 5, us, 32 x 8 heads, 1 to 2000
// keys, 8-bit: d = 64, 16 rows 26.6, 25.8; 32 rows 42.0, 40.2; 128 rows 49.6, 51.7; d = 128,
// 8 rows 26.4, 25.7; 16 rows 34.5, 34.8; 128 rows 66.0, 67.5.  bf16 behind a prefix of 512:
// d = 64, 1 row 21.5, 21.3; 8 rows 24.0, 23.1; 32 rows 40.8, 38.9; d = 128, 1 row 35.4, 35.5;
// 16 rows 39.4, 40.6.
inline int piece_tiles(int d, bool q8, int tile_rows) {
  return q8 && d == 64 && tile_rows == 8 ? 5 : 3;
}

// Query rows per unit for `rows` query rows per KV head.  Up to 16 (32 at d = 64) go
// through mma.m16n8k16 (attn_decode_rows.cu), the smallest of its tiles that holds them;
// for more, tcgen05 tiles of 128 rows are faster.  16 sequences x 8 KV heads x 16384
// keys in 8 bits, through m16n8k16 and through tcgen05, us: d = 128, 16 rows 112 and 196,
// 17 to 32 rows 279 and 196; d = 64, 16 rows 81 and 170, 17 to 32 rows 128 and 170.
inline int decode_tile_rows(int d, long long rows) {
  if (rows <= 8) return 8;
  if (rows <= 16) return 16;
  return d == 64 && rows <= 32 ? 32 : 128;
}

}  // namespace attn
