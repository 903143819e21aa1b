// fa2_paged_fp8.h -- declarations shared by the translation units of the 8-bit
// paged cache.  Not part of the public interface.
#pragma once

#include "fa2_paged.h"

namespace fa2 {

// One of K and V: 16-bit rows [total][heads][d] (strides in 16-byte units), codes
// [page][head][row][d] (strides in 8-byte units), exponents [page][head][row].
struct PagedFp8Side {
  uint4* rows;
  uint2* codes;
  uint8_t* exps;
  long long row_rs, row_hs;                // token, head
  long long code_ps, code_hs, code_rs;     // page, head, row of a page
  long long exp_ps, exp_hs;                // page, head (bytes)
};

struct PagedFp8RowsArgs {
  PagedFp8Side k, v;
  const int* slots;
  uint32_t* status;
  int total, heads, num_slots, page_size;
  int head_dim;
  unsigned page_magic, page_shift;   // as PagedParams
  bool bf16;
};

int launch_paged_append_fp8(const PagedFp8RowsArgs& a, cudaStream_t stream);
int launch_paged_read_fp8(const PagedFp8RowsArgs& a, cudaStream_t stream);

// Query rows of a tile, at most.
constexpr int kPagedFp8Rows = 32;

// Everything of an attention call on 8-bit rows.  p: as the 16-bit kernel's, with
// p.group query heads of each of p.heads_kv parts of K/V heads (`parts` of one).
struct PagedFp8Params {
  PagedParams p;
  const void* q;             // 16-bit [total_q][heads][d] by strides (elements)
  long long q_rs, q_hs;
  const uint8_t* k_exps;     // [page][head][row], strides in bytes
  const uint8_t* v_exps;
  long long k_exp_ps, k_exp_hs, v_exp_ps, v_exp_hs;
  int parts;                 // a K/V head's query heads are cut into this many parts of p.group
  float scale_log2;          // scale * log2 e, signed
  int bf16;
};

struct PagedFp8LaunchArgs {
  CUtensorMap tm_k, tm_v;    // (row bytes, 8 rows, d / 128 column blocks, then as PagedSide)
  PagedFp8Params a;
  bool many;                 // a sequence may have several query tiles, or the line 2^31 key tiles
  cudaStream_t stream;
};

int launch_paged_fp8_d64(const PagedFp8LaunchArgs& a);
int launch_paged_fp8_d128(const PagedFp8LaunchArgs& a);
int launch_paged_fp8_d256(const PagedFp8LaunchArgs& a);

}  // namespace fa2
