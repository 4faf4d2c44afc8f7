// Launch parameters of the shared-prefix kernel, shared by host and device.
#pragma once

#include <cstdint>

namespace attn {

// Query rows of one KV head: B * G of them (G = Hq / Hkv * Lq), row (b, rr) at flat
// output row (b * Hkv + hkv) * G + rr.  They are cut into `tiles` tiles of at most
// 128 rows: G <= 128: nb whole sequences each (nb = 128 / G); G > 128: 128 rows of
// one sequence (per_seq tiles each).
struct PrefixParams {
  float* ws_o;    // fp32 [nsplit, nrows, d] normalised partial outputs
  float* ws_lse;  // fp32 [nsplit, nrows]
  int* err;
  const int32_t* prefix_table;  // page ids of the prefix, or null (contiguous [Hkv, Lp, d])
  long long nrows;              // B * Hq * Lq
  int B, Hkv, G, Lp;
  int nb, per_seq, tiles, pairs;  // pairs = ceil(tiles / 2)
  int box_rows;                   // rows of a Q box: nb * G, or 128
  int chunk, nsplit;              // keys per split (multiple of 128)
  int page_size, num_pages;
  float scale_log2;
};

}  // namespace attn
