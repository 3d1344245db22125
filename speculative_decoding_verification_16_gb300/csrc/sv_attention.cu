// sv_attention.cu -- attention of a chunk of new tokens over a paged cache
// (include/spec_verify_serve.h).
#include <cuda_bf16.h>
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
};

// Request r's rows and length.  Rows out of range: l = -1.  A length out of range,
// or more rows than max_len: no key is seen, so that the rows become zeros.  *bad is
// raised for both.
struct Span {
  int32_t row0, l, seq;
};
__device__ __forceinline__ Span span_of(const AttnArgs& a, int r, bool* bad = nullptr) {
  Span s;
  s.row0 = a.row_offsets[r];
  const int32_t end = a.row_offsets[r + 1];
  s.seq = a.seq_lens[r];
  const bool rows = s.row0 >= 0 && end >= s.row0 && end <= a.n_rows;
  const bool keys = rows && end - s.row0 <= a.max_len && s.seq >= 0 &&
                    s.seq <= static_cast<int64_t>(a.table_width) * a.page;
  s.l = rows ? end - s.row0 : -1;
  if (!keys) s.seq = 0;
  if (bad != nullptr) *bad |= !keys;
  return s;
}

}  // namespace serve
}  // namespace sv

#include "sv_attn_fma.cuh"

namespace sv {
namespace serve {
namespace {

constexpr size_t round256(size_t n) { return (n + 255) / 256 * 256; }
constexpr size_t kRecordBytes = round256(sizeof(AttnRecord) * kMaxWorkers);
constexpr size_t kMlBytes = sizeof(float2) * 2 * kMaxWorkers * kRows;

int padded(int head_dim) { return head_dim <= 64 ? 64 : head_dim <= 128 ? 128 : 256; }

size_t workspace_bytes_of(int dtype, int head_dim) {
  const size_t dp = padded(head_dim);
  if (dtype == SV_FP32)
    return kRecordBytes + sizeof(float2) * 2 * kMaxWorkers * kFmaRows +
           sizeof(float) * 2 * kMaxWorkers * kFmaRows * dp;
  return kRecordBytes + kMlBytes + sizeof(float) * 2 * kMaxWorkers * kRows * (dp < 128 ? dp : 128);
}

using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                 const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                 const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                 CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiled encode_tiled() {
  static const EncodeTiled fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult found = cudaDriverEntryPointSymbolNotFound;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                         &found) != cudaSuccess ||
        found != cudaDriverEntryPointSuccess)
      p = nullptr;
    return reinterpret_cast<EncodeTiled>(p);
  }();
  return fn;
}

// A cache as (head_dim, token of a page, head, page), copied in boxes of 64
// columns and `box` tokens.
bool encode_cache(CUtensorMap* map, const void* base, const AttnArgs& a, int kv_heads, int box) {
  const cuuint64_t dims[4] = {static_cast<cuuint64_t>(a.dim), static_cast<cuuint64_t>(a.page),
                              static_cast<cuuint64_t>(kv_heads),
                              static_cast<cuuint64_t>(a.num_blocks)};
  cuuint64_t strides[3] = {static_cast<cuuint64_t>(a.token), static_cast<cuuint64_t>(a.head),
                           static_cast<cuuint64_t>(a.block)};
  for (int i = 0; i < 3; ++i)
    if (dims[i + 1] == 1) strides[i] = 16;  // never stepped along
  const cuuint32_t boxes[4] = {64, static_cast<cuuint32_t>(box), 1, 1}, one[4] = {1, 1, 1, 1};
  const EncodeTiled fn = encode_tiled();
  return fn != nullptr &&
         fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base), dims, strides, boxes,
            one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Joins the items that `grid` workers were given in parts.
template <int MR, int DP, bool F32>
int join(const MmaArgs& p, int grid, int64_t items, int64_t joins, cudaStream_t st) {
  if (grid == 1 || p.whole) return SV_OK;  // no item is cut
  Device d;
  const int rc = device(&d);
  if (rc != SV_OK) return rc;
  // few items in many parts: four threads a column take a part of them each (one
  // request's 16 tokens, 32/8 heads of 128, over 16,000 keys 27 us a call against 37; over
  // 4,000, where an item has some 20 parts, 15.7 against 14.7); many items in two parts:
  // more and smaller blocks (32 requests of mixed contexts 158 us against 170)
  if (grid >= 8 * items)
    return launch(attn_combine_kernel<MR, DP, 4, F32>,
                  dim3(static_cast<unsigned>(std::min<int64_t>(joins, 4 * d.sms))),
                  4 * combine_group(DP), 0, 1, true, st, p, grid);
  return launch(attn_combine_kernel<MR, DP, 1, F32>,
                dim3(static_cast<unsigned>(std::min<int64_t>(joins, 16 * d.sms))), combine_group(DP),
                0, 1, true, st, p, grid);
}

template <int NS, int DP>
int launch_mma(const MmaArgs& p, int grid, int64_t items, int64_t joins, const CUtensorMap& km,
               const CUtensorMap& vm, cudaStream_t st) {
  constexpr int threads = attn_threads(NS), smem = attn_smem(NS, DP);
  int rc = p.box > 0
               ? launch(attn_mma_kernel<NS, DP, true>, dim3(grid), threads, smem, 1, false, st, p, km, vm)
               : launch(attn_mma_kernel<NS, DP, false>, dim3(grid), threads, smem, 1, false, st, p, km, vm);
  return rc != SV_OK ? rc : join<NS * kRows, DP, false>(p, grid, items, joins, st);
}

// What a call's sizes bound: the row tiles' items and their key tiles.
struct Bounds {
  int64_t items, joins;
  int grid;
};
Bounds bounds(MmaArgs* p, int tile_rows, int64_t most) {
  const AttnArgs& a = p->a;
  const int64_t rows = std::min<int64_t>(a.max_len, a.n_rows) * a.group;
  const int64_t keys = static_cast<int64_t>(a.table_width) * a.page;
  // items of at most four tiles are not cut: the parts' latency and the second
  // launch would cost what they save
  p->whole = keys <= 4 * kTile;
  Bounds b;
  b.items = (rows + tile_rows - 1) / tile_rows * a.B * p->kv_heads;
  b.grid = static_cast<int>(
      std::min(most, b.items * (p->whole ? 1 : (keys + kTile - 1) / kTile)));
  // row groups of the items that can be cut: a block each
  b.joins = std::min<int64_t>(b.items, b.grid - 1) *
            ((std::min<int64_t>(rows, tile_rows) + kCombineRows - 1) / kCombineRows);
  return b;
}

int run_mma(const AttnArgs& a, int kv_heads, void* workspace, cudaStream_t st) {
  Device d;
  const int rc = device(&d);
  if (rc != SV_OK) return rc;
  const int dp = padded(a.dim);
  char* ws = static_cast<char*>(workspace);
  MmaArgs p{a, kv_heads, 0, false, reinterpret_cast<AttnRecord*>(ws),
            reinterpret_cast<float2*>(ws + kRecordBytes),
            reinterpret_cast<float4*>(ws + kRecordBytes + kMlBytes)};
  // whole page pieces by tensor copies where pages hold a number of them and
  // the strides fit a tensor map
  p.box = a.page % 64 == 0 ? 64 : a.page == 8 || a.page == 16 || a.page == 32 ? a.page : 0;
  for (int64_t s : {a.block, a.token, a.head})
    if (s >= (int64_t{1} << 40)) p.box = 0;
  if ((a.block == 0 && a.num_blocks > 1) || (a.token == 0 && a.page > 1) ||
      (a.head == 0 && kv_heads > 1))
    p.box = 0;
  CUtensorMap km{}, vm{};
  if (p.box > 0 && (!encode_cache(&km, a.k, a, kv_heads, p.box) ||
                    !encode_cache(&vm, a.v, a, kv_heads, p.box)))
    return SV_ERR_CUDA;
  const int64_t rows = std::min<int64_t>(a.max_len, a.n_rows) * a.group;
  const int ns = rows > kRows && dp <= 128 ? 2 : 1, per_sm = attn_per_sm(ns, dp);
  const Bounds b = bounds(&p, ns * kRows, std::min(per_sm * d.sms, per_sm * kMaxWorkers / 2));
  if (dp == 256) return launch_mma<1, 256>(p, b.grid, b.items, b.joins, km, vm, st);
  if (ns == 1)
    return dp == 64 ? launch_mma<1, 64>(p, b.grid, b.items, b.joins, km, vm, st)
                    : launch_mma<1, 128>(p, b.grid, b.items, b.joins, km, vm, st);
  return dp == 64 ? launch_mma<2, 64>(p, b.grid, b.items, b.joins, km, vm, st)
                  : launch_mma<2, 128>(p, b.grid, b.items, b.joins, km, vm, st);
}

template <int DP>
int launch_fma(const MmaArgs& p, const Bounds& b, cudaStream_t st) {
  const int rc =
      launch(attn_fma_kernel<DP>, dim3(b.grid), kFmaThreads, fma_smem(DP), 1, false, st, p);
  return rc != SV_OK ? rc : join<kFmaRows, DP, true>(p, b.grid, b.items, b.joins, st);
}

int run_fma(const AttnArgs& a, int kv_heads, void* workspace, cudaStream_t st) {
  Device d;
  const int rc = device(&d);
  if (rc != SV_OK) return rc;
  char* ws = static_cast<char*>(workspace);
  MmaArgs p{a, kv_heads, 0, false, reinterpret_cast<AttnRecord*>(ws),
            reinterpret_cast<float2*>(ws + kRecordBytes),
            reinterpret_cast<float4*>(ws + kRecordBytes +
                                      sizeof(float2) * 2 * kMaxWorkers * kFmaRows)};
  // shared memory holds one CTA an SM for heads above 128, else two
  const int dp = padded(a.dim), per_sm = dp == 256 ? 1 : 2;
  const Bounds b = bounds(&p, kFmaRows, std::min(per_sm * d.sms, kMaxWorkers));
  return dp == 64    ? launch_fma<64>(p, b, st)
         : dp == 128 ? launch_fma<128>(p, b, st)
                     : launch_fma<256>(p, b, st);
}

}  // namespace
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
  if (dtype != SV_BF16 && dtype != SV_FP32) return SV_ERR_DTYPE;
  const int es = dtype == SV_BF16 ? 2 : 4;
  if (B < 1 || n_rows < 0 || max_len < 1 || heads < 1 || kv_heads < 1 || heads % kv_heads != 0 ||
      head_dim < 1 || num_blocks < 1 || page_size < 1 || table_width < 1 ||
      table_stride < table_width || !std::isfinite(scale))
    return SV_ERR_ARG;
  if (head_dim % 8 != 0 || head_dim > SV_ATTN_MAX_HEAD_DIM) return SV_ERR_UNSUPPORTED;
  if (static_cast<int64_t>(table_width) * page_size > INT32_MAX / 2 ||
      static_cast<int64_t>(n_rows) * heads > INT32_MAX)
    return SV_ERR_UNSUPPORTED;
  if (n_rows == 0) return SV_OK;  // an empty tensor has no address
  if (query == nullptr || key_cache == nullptr || value_cache == nullptr || out == nullptr ||
      block_table == nullptr || seq_lens == nullptr || row_offsets == nullptr)
    return SV_ERR_ARG;
  for (const void* p : {query, key_cache, value_cache, static_cast<const void*>(out)})
    if (!aligned_to(p, 16)) return SV_ERR_ARG;
  // a dimension of one is never stepped along, whatever its stride says
  for (int64_t s : {n_rows > 1 ? q_row_stride : 0, heads > 1 ? q_head_stride : 0,
                    num_blocks > 1 ? block_stride : 0, page_size > 1 ? token_stride : 0,
                    kv_heads > 1 ? head_stride : 0, n_rows > 1 ? o_row_stride : 0,
                    heads > 1 ? o_head_stride : 0})
    if (s < 0 || s * es % 16 != 0) return SV_ERR_ARG;
  if (!aligned_to(block_table, 4) || !aligned_to(seq_lens, 4) || !aligned_to(row_offsets, 4) ||
      !null_or_aligned(out_lse, 4) || !null_or_aligned(dev_error, 4))
    return SV_ERR_ARG;
  if (workspace == nullptr || !aligned_to(workspace, 256) ||
      workspace_bytes < spec_verify_attention_workspace_size(n_rows, heads, head_dim, dtype))
    return SV_ERR_WORKSPACE;
  // the largest scales leave fp32 here: inf * 0 would be NaN where the score is 0
  const float c = std::min(std::max(scale * kLog2e, -FLT_MAX), FLT_MAX);
  const AttnArgs a{static_cast<const char*>(query), q_row_stride * es, q_head_stride * es,
                   static_cast<const char*>(key_cache), static_cast<const char*>(value_cache),
                   block_stride * es, token_stride * es, head_stride * es, block_table,
                   table_stride, table_width, seq_lens, row_offsets, B, n_rows, max_len, heads,
                   heads / kv_heads, head_dim, num_blocks, page_size,
                   // no window where it holds every key; a row before the first key would
                   // take position - window below 32 bits
                   window >= static_cast<int64_t>(table_width) * page_size ? 0 : window,
                   // scale 0: masked scores stay -inf, and no finite product weighs: 2^128 2^-149
                   // is nothing beside 1
                   c == 0.0f ? 0x1p-149f : c,
                   static_cast<char*>(out), o_row_stride * es, o_head_stride * es, out_lse,
                   dev_error, FastDiv::by(static_cast<uint32_t>(heads / kv_heads)),
                   FastDiv::by(static_cast<uint32_t>(page_size))};
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (dtype == SV_BF16) return run_mma(a, kv_heads, workspace, st);
  return run_fma(a, kv_heads, workspace, st);
}

}  // extern "C"
