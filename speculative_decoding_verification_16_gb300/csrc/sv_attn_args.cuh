// sv_attn_args.cuh -- what the attention kernels of a paged cache share: the
// arguments of a call, a request's span, and the host's choice of items and workers.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cfloat>
#include <cmath>
#include <cstdint>

#include "sv_host.cuh"
#include "sv_ptx.cuh"

namespace sv {
namespace serve {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kInf = __builtin_huge_valf();

struct AttnArgs {
  const char* q;
  int64_t q_row, q_head;  // bytes
  const char *k, *v;
  int64_t block, token, head;  // bytes
  const int32_t* table;
  int64_t table_stride;
  int32_t table_width;
  const int32_t *seq_lens, *row_offsets;
  int32_t B, n_rows, max_len, heads, group, dim, num_blocks, page, window;
  float scale2;  // scale * log2(e): scores in powers of two
  char* out;
  int64_t o_row, o_head;  // bytes
  float* lse;
  int32_t* dev_error;
  FastDiv by_group, by_page;
  // e4m3 caches: exponents, and the strides above are those of the codes
  const int8_t *k_exps, *v_exps;
  int32_t e_block, e_token, e_head;
  // trees: of every row the rows of its request that it sees; positions may be NULL
  const uint32_t* mask;
  int32_t mask_words;
  const int32_t* positions;
};

// Request r's rows and length.  Rows out of range: l = -1.  A length out of range (of
// a tree: shorter than its rows too), or more rows than max_len: no key is seen, so
// that the rows become zeros.  *bad is raised for both.  EXT: there may be masks.
struct Span {
  int32_t row0, l, seq;
};
template <bool EXT>
__device__ __forceinline__ Span span_of(const AttnArgs& a, int r, bool* bad = nullptr) {
  Span s;
  s.row0 = a.row_offsets[r];
  const int32_t end = a.row_offsets[r + 1];
  s.seq = a.seq_lens[r];
  const bool rows = s.row0 >= 0 && end >= s.row0 && end <= a.n_rows;
  const bool keys = rows && end - s.row0 <= a.max_len && s.seq >= (EXT && a.mask != nullptr ? end - s.row0 : 0) &&
                    s.seq <= static_cast<int64_t>(a.table_width) * a.page;
  s.l = rows ? end - s.row0 : -1;
  if (!keys) s.seq = 0;
  if (bad != nullptr) *bad |= !keys;
  return s;
}

// The arguments of an attention entry point, as given.
struct AttnCall {
  const void *query, *key_cache, *value_cache;
  int64_t q_row_stride, q_head_stride, block_stride, token_stride, head_stride;
  const int8_t *key_exps, *value_exps;
  int64_t e_block_stride, e_token_stride, e_head_stride;
  const int32_t* block_table;
  int64_t table_stride;
  int32_t table_width;
  const int32_t *seq_lens, *row_offsets, *tree_mask, *positions;
  int32_t mask_words, B, n_rows, max_len, heads, kv_heads, head_dim, num_blocks, page_size;
  int32_t dtype, cache_dtype;
  float scale;
  int32_t window;
  void* out;
  int64_t o_row_stride, o_head_stride;
  float* out_lse;
  int32_t* dev_error;
  void* workspace;
  size_t workspace_bytes;
};
// Checks a call (SV_ERR_*) and, where it has rows, gives the kernels' arguments.
int attention_args(const AttnCall& c, AttnArgs* out);

}  // namespace serve
}  // namespace sv
