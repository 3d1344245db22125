// sv_attn_host.cuh -- the host's side of the attention kernels: workspace, tensor
// maps, the number of workers, launches.  Each translation unit instantiates the
// kernels that its entry point calls; the join of cut items is in sv_attention.cu.
#pragma once

#include <algorithm>
#include <cstdint>

#include "sv_attn_args.cuh"
#include "sv_attn_fma.cuh"
#include "sv_attn_mma.cuh"

namespace sv {
namespace serve {

// Joins the items that `grid` workers were given in parts of `mr` rows.
int join(const MmaArgs& p, int mr, int dp, bool f32, int grid, int64_t items, int64_t joins,
         cudaStream_t st);

namespace {

constexpr size_t round256(size_t n) { return (n + 255) / 256 * 256; }
constexpr size_t kRecordBytes = round256(sizeof(AttnRecord) * kMaxWorkers);
constexpr size_t kMlBytes = sizeof(float2) * 2 * kMaxWorkers * kRows;

int padded(int head_dim) { return head_dim <= 64 ? 64 : head_dim <= 128 ? 128 : 256; }

[[maybe_unused]] size_t workspace_bytes_of(int dtype, int head_dim) {
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

// A cache as (head_dim, token of a page, head, page), copied in boxes of 64 columns (of
// codes 128; of heads up to 64 dimensions 64, not swizzled) and `box` tokens.
bool encode_cache(CUtensorMap* map, const void* base, const AttnArgs& a, int kv_heads, int box, bool codes) {
  const cuuint64_t dims[4] = {static_cast<cuuint64_t>(a.dim), static_cast<cuuint64_t>(a.page),
                              static_cast<cuuint64_t>(kv_heads),
                              static_cast<cuuint64_t>(a.num_blocks)};
  cuuint64_t strides[3] = {static_cast<cuuint64_t>(a.token), static_cast<cuuint64_t>(a.head),
                           static_cast<cuuint64_t>(a.block)};
  for (int i = 0; i < 3; ++i)
    if (dims[i + 1] == 1) strides[i] = 16;  // never stepped along
  const bool wide = !codes || a.dim > 64;
  const cuuint32_t boxes[4] = {codes && wide ? 128u : 64u, static_cast<cuuint32_t>(box), 1, 1},
                   one[4] = {1, 1, 1, 1};
  const EncodeTiled fn = encode_tiled();
  return fn != nullptr &&
         fn(map, codes ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4,
            const_cast<void*>(base), dims, strides, boxes, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
            wide ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
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

template <int NS, int DP, int SRC, bool TREE>
int launch_mma(const MmaArgs& p, int grid, int64_t items, int64_t joins, const CUtensorMap& km,
               const CUtensorMap& vm, cudaStream_t st) {
  constexpr int threads = attn_threads(NS, DP, SRC), smem = attn_smem(NS, DP);
  const int rc = launch(attn_mma_kernel<NS, DP, SRC, TREE>, dim3(grid), threads, smem, 1, false, st,
                        p, km, vm);
  return rc != SV_OK ? rc : join(p, NS * kRows, DP, false, grid, items, joins, st);
}

template <int SRC, bool TREE>
int run_mma_from(const MmaArgs& p, const CUtensorMap& km, const CUtensorMap& vm, int sms, cudaStream_t st) {
  MmaArgs x = p;
  const int dp = padded(p.a.dim);
  const int64_t rows = std::min<int64_t>(p.a.max_len, p.a.n_rows) * p.a.group;
  const int ns = rows > kRows && dp <= 128 ? 2 : 1, per_sm = attn_per_sm(ns, dp);
  const Bounds b = bounds(&x, ns * kRows, std::min(per_sm * sms, per_sm * kMaxWorkers / 2));
  if (dp == 256) return launch_mma<1, 256, SRC, TREE>(x, b.grid, b.items, b.joins, km, vm, st);
  if (ns == 1)
    return dp == 64 ? launch_mma<1, 64, SRC, TREE>(x, b.grid, b.items, b.joins, km, vm, st)
                    : launch_mma<1, 128, SRC, TREE>(x, b.grid, b.items, b.joins, km, vm, st);
  return dp == 64 ? launch_mma<2, 64, SRC, TREE>(x, b.grid, b.items, b.joins, km, vm, st)
                  : launch_mma<2, 128, SRC, TREE>(x, b.grid, b.items, b.joins, km, vm, st);
}

// What an item of this many rows costs beside its tiles, in tiles.  32 requests over 512 to
// 32,768 (trees 16,384) tokens, us at 2 / 4 / 6 / 8 / 10 / 12, codes of 8 rows an item 137 /
// 131 / 133 / 134 / 135 / 139, 32 rows 153 / 143 / 135 / 135 / 136 / 139, 64 rows 164 / 150 /
// 143 / 142 / 142 / 146, 128 rows 192 / 181 / 172 / 169 / 170 / 172, 256 rows in two streams
// 335 / 305 / 279 / 266 / 255 / 253; bf16 trees of up to 32 rows 91 / 91 / 92 / 92 / 93 / 94,
// 128 rows 103 / 101 / 101 / 102 / 103 / 104, 256 rows 145 / 131 / 126 / 122 / 124 / 127.  So
// few rows want 4 to 6, many 8 to 12; about 64 rows either will do.
int item_cost(int64_t rows) { return rows > 32 ? 10 : 6; }

// E4M3: the caches hold codes and exponents; TREE: rows see what their masks name.
template <bool E4M3, bool TREE>
int run_mma(const AttnArgs& a, int kv_heads, void* workspace, cudaStream_t st) {
  Device d;
  const int rc = device(&d);
  if (rc != SV_OK) return rc;
  char* ws = static_cast<char*>(workspace);
  MmaArgs p{a, kv_heads, 0, false, 
            E4M3 || TREE ? item_cost(std::min<int64_t>(a.max_len, a.n_rows) * a.group) : 0, reinterpret_cast<AttnRecord*>(ws),
            reinterpret_cast<float2*>(ws + kRecordBytes),
            reinterpret_cast<float4*>(ws + kRecordBytes + kMlBytes)};
  CUtensorMap km{}, vm{};
  // whole page pieces by tensor copies where pages hold a number of them and
  // the strides fit a tensor map
  p.box = a.page % 64 == 0 ? 64 : a.page == 8 || a.page == 16 || a.page == 32 ? a.page : 0;
  for (int64_t s : {a.block, a.token, a.head})
    if (s >= (int64_t{1} << 40)) p.box = 0;
  if ((a.block == 0 && a.num_blocks > 1) || (a.token == 0 && a.page > 1) ||
      (a.head == 0 && kv_heads > 1))
    p.box = 0;
  if (p.box == 0) return run_mma_from<E4M3 ? kCodeRows : kRowCopies, TREE>(p, km, vm, d.sms, st);
  if (!encode_cache(&km, a.k, a, kv_heads, p.box, E4M3) ||
      !encode_cache(&vm, a.v, a, kv_heads, p.box, E4M3))
    return SV_ERR_CUDA;
  return run_mma_from<E4M3 ? kCodeTensor : kTensorCopies, TREE>(p, km, vm, d.sms, st);
}

template <int DP, bool TREE>
int launch_fma(const MmaArgs& p, const Bounds& b, cudaStream_t st) {
  const int rc =
      launch(attn_fma_kernel<DP, TREE>, dim3(b.grid), kFmaThreads, fma_smem(DP), 1, false, st, p);
  return rc != SV_OK ? rc : join(p, kFmaRows, DP, true, b.grid, b.items, b.joins, st);
}

template <bool TREE>
int run_fma(const AttnArgs& a, int kv_heads, void* workspace, cudaStream_t st) {
  Device d;
  const int rc = device(&d);
  if (rc != SV_OK) return rc;
  char* ws = static_cast<char*>(workspace);
  MmaArgs p{a, kv_heads, 0, false, 0, reinterpret_cast<AttnRecord*>(ws),
            reinterpret_cast<float2*>(ws + kRecordBytes),
            reinterpret_cast<float4*>(ws + kRecordBytes +
                                      sizeof(float2) * 2 * kMaxWorkers * kFmaRows)};
  // shared memory holds one CTA an SM for heads above 128, else two
  const int dp = padded(a.dim), per_sm = dp == 256 ? 1 : 2;
  const Bounds b = bounds(&p, kFmaRows, std::min(per_sm * d.sms, kMaxWorkers));
  return dp == 64    ? launch_fma<64, TREE>(p, b, st)
         : dp == 128 ? launch_fma<128, TREE>(p, b, st)
                     : launch_fma<256, TREE>(p, b, st);
}

}  // namespace
}  // namespace serve
}  // namespace sv
