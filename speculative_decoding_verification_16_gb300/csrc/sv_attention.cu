// sv_attention.cu -- attention of a chunk of new tokens over a paged cache
// (include/spec_verify_serve.h).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cfloat>
#include <cmath>
#include <cstdint>

#include "sv_attn_host.cuh"

namespace sv {
namespace serve {

namespace {

template <int MR, int DP, bool F32, bool CODES>
int join_of(const MmaArgs& p, int grid, int64_t items, int64_t joins, cudaStream_t st) {
  if (grid == 1 || p.whole) return SV_OK;  // no item is cut
  Device d;
  const int rc = device(&d);
  if (rc != SV_OK) return rc;
  // few items in many parts: four threads a column take a part of them each (one
  // request's 16 tokens, 32/8 heads of 128, over 16,000 keys 27 us a call against 37; over
  // 4,000, where an item has some 20 parts, 15.7 against 14.7); many items in two parts:
  // more and smaller blocks (32 requests of mixed contexts 158 us against 170)
  if (grid >= 8 * items)
    return launch(attn_combine_kernel<MR, DP, 4, F32, CODES>,
                  dim3(static_cast<unsigned>(std::min<int64_t>(joins, 4 * d.sms))),
                  4 * combine_group(DP), 0, 1, true, st, p, grid);
  return launch(attn_combine_kernel<MR, DP, 1, F32, CODES>,
                dim3(static_cast<unsigned>(std::min<int64_t>(joins, 16 * d.sms))), combine_group(DP),
                0, 1, true, st, p, grid);
}

template <bool CODES>
int join_mma(const MmaArgs& p, int mr, int dp, int grid, int64_t items, int64_t joins, cudaStream_t st) {
  if (dp == 256) return join_of<kRows, 256, false, CODES>(p, grid, items, joins, st);
  if (mr == kRows)
    return dp == 64 ? join_of<kRows, 64, false, CODES>(p, grid, items, joins, st)
                    : join_of<kRows, 128, false, CODES>(p, grid, items, joins, st);
  return dp == 64 ? join_of<2 * kRows, 64, false, CODES>(p, grid, items, joins, st)
                  : join_of<2 * kRows, 128, false, CODES>(p, grid, items, joins, st);
}

}  // namespace

int join(const MmaArgs& p, int mr, int dp, bool f32, int grid, int64_t items, int64_t joins,
         cudaStream_t st) {
  if (f32)
    return dp == 64    ? join_of<kFmaRows, 64, true, false>(p, grid, items, joins, st)
           : dp == 128 ? join_of<kFmaRows, 128, true, false>(p, grid, items, joins, st)
                       : join_of<kFmaRows, 256, true, false>(p, grid, items, joins, st);
  return p.a.k_exps != nullptr ? join_mma<true>(p, mr, dp, grid, items, joins, st)
                               : join_mma<false>(p, mr, dp, grid, items, joins, st);
}

// The checks of a call and the kernels' arguments.
int attention_args(const AttnCall& c, AttnArgs* out) {
  if (c.dtype != SV_BF16 && c.dtype != SV_FP32) return SV_ERR_DTYPE;
  const bool codes = c.cache_dtype == SV_E4M3;
  if (codes ? c.dtype != SV_BF16 : c.cache_dtype != c.dtype) return SV_ERR_DTYPE;
  const int es = c.dtype == SV_BF16 ? 2 : 4, cs = codes ? 1 : es;
  if (c.B < 1 || c.n_rows < 0 || c.max_len < 1 || c.heads < 1 || c.kv_heads < 1 ||
      c.heads % c.kv_heads != 0 || c.head_dim < 1 || c.num_blocks < 1 || c.page_size < 1 ||
      c.table_width < 1 || c.table_stride < c.table_width || !std::isfinite(c.scale))
    return SV_ERR_ARG;
  if (c.tree_mask != nullptr && c.mask_words < (c.max_len - 1) / 32 + 1) return SV_ERR_ARG;
  if (c.head_dim % (codes ? 16 : 8) != 0 || c.head_dim > SV_ATTN_MAX_HEAD_DIM)
    return SV_ERR_UNSUPPORTED;
  if (static_cast<int64_t>(c.table_width) * c.page_size > INT32_MAX / 2 ||
      static_cast<int64_t>(c.n_rows) * c.heads > INT32_MAX)
    return SV_ERR_UNSUPPORTED;
  if (c.n_rows == 0) return SV_OK;  // an empty tensor has no address
  if (c.query == nullptr || c.key_cache == nullptr || c.value_cache == nullptr ||
      c.out == nullptr || c.block_table == nullptr || c.seq_lens == nullptr ||
      c.row_offsets == nullptr || (codes && (c.key_exps == nullptr || c.value_exps == nullptr)))
    return SV_ERR_ARG;
  // the window of a tree's row starts from its position
  if (c.tree_mask != nullptr && c.window > 0 && c.positions == nullptr) return SV_ERR_ARG;
  for (const void* p : {c.query, c.key_cache, c.value_cache, static_cast<const void*>(c.out)})
    if (!aligned_to(p, 16)) return SV_ERR_ARG;
  // a dimension of one is never stepped along, whatever its stride says
  for (int64_t s : {c.n_rows > 1 ? c.q_row_stride : 0, c.heads > 1 ? c.q_head_stride : 0,
                    c.n_rows > 1 ? c.o_row_stride : 0, c.heads > 1 ? c.o_head_stride : 0})
    if (s < 0 || s * es % 16 != 0) return SV_ERR_ARG;
  for (int64_t s : {c.num_blocks > 1 ? c.block_stride : 0, c.page_size > 1 ? c.token_stride : 0,
                    c.kv_heads > 1 ? c.head_stride : 0})
    if (s < 0 || s * cs % 16 != 0) return SV_ERR_ARG;
  if (codes)
    for (int64_t s : {c.num_blocks > 1 ? c.e_block_stride : 0, c.page_size > 1 ? c.e_token_stride : 0,
                      c.kv_heads > 1 ? c.e_head_stride : 0}) {
      if (s < 0) return SV_ERR_ARG;
      if (s > INT32_MAX) return SV_ERR_UNSUPPORTED;
    }
  if (!aligned_to(c.block_table, 4) || !aligned_to(c.seq_lens, 4) ||
      !aligned_to(c.row_offsets, 4) || !null_or_aligned(c.out_lse, 4) ||
      !null_or_aligned(c.dev_error, 4) || !null_or_aligned(c.tree_mask, 4) ||
      !null_or_aligned(c.positions, 4))
    return SV_ERR_ARG;
  if (c.workspace == nullptr || !aligned_to(c.workspace, 256) ||
      c.workspace_bytes < workspace_bytes_of(c.dtype, c.head_dim))
    return SV_ERR_WORKSPACE;
  // the largest scales leave fp32 here: inf * 0 would be NaN where the score is 0
  const float f = std::min(std::max(c.scale * kLog2e, -FLT_MAX), FLT_MAX);
  *out = AttnArgs{static_cast<const char*>(c.query), c.q_row_stride * es, c.q_head_stride * es,
                  static_cast<const char*>(c.key_cache), static_cast<const char*>(c.value_cache),
                  c.block_stride * cs, c.token_stride * cs, c.head_stride * cs, c.block_table,
                  c.table_stride, c.table_width, c.seq_lens, c.row_offsets, c.B, c.n_rows,
                  c.max_len, c.heads, c.heads / c.kv_heads, c.head_dim, c.num_blocks, c.page_size,
                  // no window where it holds every key; a row before the first key would
                  // take position - window below 32 bits
                  c.window >= static_cast<int64_t>(c.table_width) * c.page_size ? 0 : c.window,
                  // scale 0: masked scores stay -inf, and no finite product weighs: 2^128 2^-149
                  // is nothing beside 1
                  f == 0.0f ? 0x1p-149f : f,
                  static_cast<char*>(c.out), c.o_row_stride * es, c.o_head_stride * es, c.out_lse,
                  c.dev_error, FastDiv::by(static_cast<uint32_t>(c.heads / c.kv_heads)),
                  FastDiv::by(static_cast<uint32_t>(c.page_size)),
                  codes ? c.key_exps : nullptr, codes ? c.value_exps : nullptr, static_cast<int32_t>(c.e_block_stride),
                  static_cast<int32_t>(c.e_token_stride), static_cast<int32_t>(c.e_head_stride),
                  reinterpret_cast<const uint32_t*>(c.tree_mask), c.mask_words, c.positions};
  return SV_OK;
}

}  // namespace serve
}  // namespace sv

extern "C" {

size_t spec_verify_attention_workspace_size(int32_t n_rows, int32_t heads, int32_t head_dim,
                                            int32_t dtype) {
  (void)n_rows, (void)heads;
  return sv::serve::workspace_bytes_of(dtype, head_dim);
}

int spec_verify_attention(const void* query, int64_t q_row_stride, int64_t q_head_stride,
                          const void* key_cache, const void* value_cache, int64_t block_stride,
                          int64_t token_stride, int64_t head_stride, const int32_t* block_table,
                          int64_t table_stride, int32_t table_width, const int32_t* seq_lens,
                          const int32_t* row_offsets, int32_t B, int32_t n_rows, int32_t max_len,
                          int32_t heads, int32_t kv_heads, int32_t head_dim, int32_t num_blocks,
                          int32_t page_size, int32_t dtype, float scale, int32_t window,
                          void* out, int64_t o_row_stride, int64_t o_head_stride, float* out_lse,
                          int32_t* dev_error, void* workspace, size_t workspace_bytes,
                          void* stream) {
  using namespace sv::serve;
  AttnCall c{};
  c.query = query, c.q_row_stride = q_row_stride, c.q_head_stride = q_head_stride;
  c.key_cache = key_cache, c.value_cache = value_cache;
  c.block_stride = block_stride, c.token_stride = token_stride, c.head_stride = head_stride;
  c.block_table = block_table, c.table_stride = table_stride, c.table_width = table_width;
  c.seq_lens = seq_lens, c.row_offsets = row_offsets;
  c.B = B, c.n_rows = n_rows, c.max_len = max_len, c.heads = heads, c.kv_heads = kv_heads;
  c.head_dim = head_dim, c.num_blocks = num_blocks, c.page_size = page_size;
  c.dtype = c.cache_dtype = dtype, c.scale = scale, c.window = window;
  c.out = out, c.o_row_stride = o_row_stride, c.o_head_stride = o_head_stride;
  c.out_lse = out_lse, c.dev_error = dev_error;
  c.workspace = workspace, c.workspace_bytes = workspace_bytes;
  AttnArgs a;
  const int rc = attention_args(c, &a);
  if (rc != SV_OK || n_rows == 0) return rc;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (dtype == SV_BF16) return run_mma<false, false>(a, kv_heads, workspace, st);
  return run_fma<false>(a, kv_heads, workspace, st);
}

}  // extern "C"
