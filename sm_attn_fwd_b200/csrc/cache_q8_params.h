// Launch parameters of the 8-bit cache kernels, shared by host and device.
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

// Decode over an 8-bit cache.
struct DecodeQ8Params {
  const void* q;  // bf16 [B, Hq, Lq, d]
  void* o;        // bf16, written when nsplit == 1
  float* lse;     // fp32, written when nsplit == 1
  float* ws_o;    // fp32 [nsplit, B*Hq*Lq, d] otherwise
  float* ws_lse;  // fp32 [nsplit, B*Hq*Lq]
  const uint8_t* k_exp;
  const uint8_t* v_exp;
  const int32_t* kv_lens;
  const int32_t* block_table;
  int* err;
  int B, Hq, Hkv, Lq, Lk, group;
  float scale_log2;
  int chunk, nsplit;
  int row_tiles;  // row tiles per (b, kv head)
  int page_size, page_shift, pages_per_seq, num_pages;
};

}  // namespace attn
