// sv_tree.cu -- trees of drafted tokens: masks and positions from parents, the
// accepted path, and its keys and values moved together
// (include/spec_verify_serve.h).
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "sv_host.cuh"
#include "sv_ptx.cuh"

namespace sv {
namespace serve {
namespace {

constexpr int kTreeRows = SV_MAX_LEN;         // most rows of a request
constexpr int kTreeWords = kTreeRows / 32;

// A request's rows, or -1 where row_offsets do not rise within [0, n_rows].
struct TreeSpan {
  int32_t row0, l;
};
__device__ __forceinline__ TreeSpan tree_span(const int32_t* row_offsets, int r, int n_rows) {
  const int32_t row0 = row_offsets[r], end = row_offsets[r + 1];
  return {row0, row0 >= 0 && end >= row0 && end <= n_rows ? end - row0 : -1};
}

// ---------------------------------------------------------------- masks and positions
//
// A CTA a request, a thread a row.  Each row starts with itself and its parent and
// doubles its reach: it takes in the mask of the highest row it knows of and goes on
// from there, log2(depth) rounds through shared memory.  Bound by latency: two rounds
// of loads, the doubling, the stores.  32 trees of up to 64 rows 4.1 us called, 256 of up
// to 256 6.2.
struct PlanArgs {
  const int32_t *parents, *seq_lens, *row_offsets;
  int32_t B, n_rows, max_len, words;
  int32_t *positions, *mask, *dev_error;
};

__global__ __launch_bounds__(kTreeRows) void tree_plan_kernel(const PlanArgs a) {
  __shared__ uint32_t bits[kTreeWords][kTreeRows];
  __shared__ int16_t up[kTreeRows], depth[kTreeRows];
  const int i = threadIdx.x, r = blockIdx.x;
  if (r >= a.B) {  // rows behind the last request
    const int end = max(0, a.row_offsets[a.B]);
    const int step = (gridDim.x - a.B) * blockDim.x;
    for (int64_t row = static_cast<int64_t>(end) + (r - a.B) * blockDim.x + i; row < a.n_rows; row += step) {
      a.positions[row] = 0;
      for (int w = 0; w < a.words; ++w) a.mask[row * a.words + w] = 0;
    }
    return;
  }
  const TreeSpan s = tree_span(a.row_offsets, r, a.n_rows);
  const int32_t seq = a.seq_lens[r];
  uint32_t err = 0;
  if (s.l < 0) {
    if (i == 0 && a.dev_error != nullptr) atomicOr(a.dev_error, SV_DEVERR_LEN);
    return;
  }
  if (s.l > a.max_len || seq < s.l) {  // not served: nothing is seen
    for (int row = i; row < s.l; row += blockDim.x) {
      a.positions[s.row0 + row] = 0;
      for (int w = 0; w < a.words; ++w) a.mask[static_cast<int64_t>(s.row0 + row) * a.words + w] = 0;
    }
    if (i == 0 && s.l > 0 && a.dev_error != nullptr) atomicOr(a.dev_error, SV_DEVERR_LEN);
    return;
  }
  const bool on = i < s.l;
  int p = on ? a.parents[s.row0 + i] : -1, d;
  if (p < -1 || p >= i) err = SV_DEVERR_TREE, p = -1;
  d = p >= 0;
  const int words = (s.l + 31) / 32;
  uint32_t m[kTreeWords];
#pragma unroll
  for (int w = 0; w < kTreeWords; ++w) m[w] = on && w == i / 32 ? 1u << i % 32 : 0;
  while (true) {  // p: the highest row that is not in m yet, or -1; d: steps up to p
#pragma unroll
    for (int w = 0; w < kTreeWords; ++w)
      if (w < words) bits[w][i] = m[w];
    up[i] = static_cast<int16_t>(p), depth[i] = static_cast<int16_t>(d);
    if (__syncthreads_or(p >= 0) == 0) break;
    if (p >= 0) {
#pragma unroll
      for (int w = 0; w < kTreeWords; ++w)
        if (w < words) m[w] |= bits[w][p];
      d += depth[p];
      p = up[p];
    }
    __syncthreads();
  }
  if (on) {
    const int64_t row = s.row0 + i;
    a.positions[row] = seq - s.l + d;
#pragma unroll
    for (int w = 0; w < kTreeWords; ++w)
      if (w < a.words) a.mask[row * a.words + w] = static_cast<int32_t>(m[w]);
    for (int w = kTreeWords; w < a.words; ++w) a.mask[row * a.words + w] = 0;
  }
  if (err != 0 && a.dev_error != nullptr) atomicOr(a.dev_error, static_cast<int32_t>(err));
}

// ---------------------------------------------------------------- the accepted path
//
// A CTA a request, a thread a row: each row whose token is the one that the target
// gave after its parent offers itself to it, the lowest wins (none where that is -1, no
// token: a draft that could not be sampled is -1 too); one thread walks down from the root.
// Bound by latency: three rounds of loads and the walk.
struct AcceptArgs {
  const int32_t *tokens, *next, *parents, *row_offsets;
  int32_t B, n_rows, max_len;
  int32_t *out_tokens, *path, *accept_len, *dev_error;
};

__global__ __launch_bounds__(kTreeRows) void tree_accept_kernel(const AcceptArgs a) {
  __shared__ int32_t child[kTreeRows], after[kTreeRows], way[kTreeRows];
  __shared__ int32_t count;
  const int i = threadIdx.x, r = blockIdx.x;
  if (r >= a.B) {  // rows behind the last request
    const int end = max(0, a.row_offsets[a.B]);
    const int step = (gridDim.x - a.B) * blockDim.x;
    for (int64_t row = static_cast<int64_t>(end) + (r - a.B) * blockDim.x + i; row < a.n_rows; row += step)
      a.out_tokens[row] = a.path[row] = -1;
    return;
  }
  const TreeSpan s = tree_span(a.row_offsets, r, a.n_rows);
  if (s.l <= 0 || s.l > a.max_len) {
    for (int row = i; row < s.l; row += blockDim.x) a.out_tokens[s.row0 + row] = a.path[s.row0 + row] = -1;
    if (i == 0) {
      a.accept_len[r] = -1;
      if (s.l != 0 && a.dev_error != nullptr) atomicOr(a.dev_error, SV_DEVERR_LEN);
    }
    return;
  }
  const bool on = i < s.l;
  const int64_t row = s.row0 + i;
  child[i] = INT32_MAX;
  int p = -1, token = 0;
  if (on) {
    after[i] = a.next[row];
    token = a.tokens[row];
    p = a.parents[row];
    if (p < -1 || p >= i) {
      if (a.dev_error != nullptr) atomicOr(a.dev_error, SV_DEVERR_TREE);
      p = -1;
    }
  }
  __syncthreads();
  if (p >= 0 && token >= 0 && token == after[p]) atomicMin(&child[p], i);
  __syncthreads();
  if (i == 0) {
    int at = 0, n = 0;
    for (; at != INT32_MAX; at = child[at]) way[n++] = at;  // rows rise: at most l
    count = n;
    a.accept_len[r] = n - 1;
  }
  __syncthreads();
  if (on) {
    a.path[row] = i < count ? way[i] : -1;
    a.out_tokens[row] = i < count ? after[way[i]] : -1;
  }
}

// ---------------------------------------------------------------- moves
//
// Row path[j] of a request moves to row j, in all layers.  Rows rise along the path,
// path[j] >= j, so a thread that takes the moves of its bytes in order of j never
// writes what a later move still reads, though sources and targets overlap.  A CTA a
// request and some layers: it lists the moves once, then its threads each own units of
// 16 bytes of a layer, four moves' loads in flight at a time.  Bound by latency: five
// rounds of dependent loads (offsets, length, path, slots, data).  With the accepted paths
// 10 us called for 8 requests in one layer, 16 for 128 requests in 32 layers.
constexpr int kMoveThreads = 256;

struct MoveArgs {
  const int32_t *path, *accept_len, *row_offsets;
  const int64_t* slots;
  int32_t B, n_rows, max_len, layers, layers_per_cta;
  char *k, *v;
  int64_t layer, block, token, head;  // bytes
  int8_t *k_exps, *v_exps;
  int64_t e_layer, e_block, e_token, e_head;
  int64_t n_slots;
  int32_t page, kv_heads, units, head_units;  // units of a row of keys, and of a head
  int32_t* dev_error;
  FastDiv by_head, by_units;
};

template <typename U>
__global__ __launch_bounds__(kMoveThreads) void tree_move_kernel(const MoveArgs a) {
  __shared__ int64_t from[kTreeRows], to[kTreeRows];          // slots
  __shared__ uint8_t ok[kTreeRows];
  __shared__ int32_t list[kTreeRows], count;
  const int tid = threadIdx.x, r = blockIdx.x;
  const TreeSpan s = tree_span(a.row_offsets, r, a.n_rows);
  const int n = a.accept_len[r];  // moves of rows 1 .. n
  if (s.l < 0 || s.l > a.max_len || n < -1 || n >= s.l) {
    if (tid == 0 && blockIdx.y == 0 && a.dev_error != nullptr) atomicOr(a.dev_error, SV_DEVERR_LEN);
    return;
  }
  if (n < 1) return;
  uint32_t err = 0;
  for (int j = tid; j <= n; j += kMoveThreads) {
    const int at = a.path[s.row0 + j], before = j > 0 ? a.path[s.row0 + j - 1] : -1;
    // 0: stays, as row 0 does wherever the path starts; 1: moves; 2: the path ends here, it
    // does not rise
    ok[j] = at <= before || at < j || at >= s.l ? 2 : at == j || j == 0 ? 0 : 1;
    if (ok[j] == 1) {
      const int64_t f = a.slots[s.row0 + at], t = a.slots[s.row0 + j];
      from[j] = f, to[j] = t;
      if (f >= a.n_slots || t >= a.n_slots) err |= SV_DEVERR_PAGE;
      if (f < 0 || t < 0 || f >= a.n_slots || t >= a.n_slots) ok[j] = 0;
    }
    if (ok[j] == 2) err |= SV_DEVERR_TREE;
  }
  __syncthreads();
  if (tid < 32) {  // the moves in order, up to where the path stops rising
    int k = 0;
    for (int base = 0; base <= n; base += 32) {
      const int j = base + tid;
      const unsigned bad = __ballot_sync(~0u, j <= n && ok[j] == 2);
      const unsigned fine = bad != 0 ? (bad & -bad) - 1 : ~0u;
      const unsigned moves = __ballot_sync(~0u, j <= n && ok[j] == 1) & fine;
      if (moves >> tid & 1) list[k + __popc(moves & ((1u << tid) - 1))] = j;
      k += __popc(moves);
      if (bad != 0) break;
    }
    if (tid == 0) count = k;
  }
  __syncthreads();
  const int moves = count;
  auto offset = [&](int64_t slot, int64_t block, int64_t token) {
    const int64_t b = slot / a.page;
    return b * block + (slot - b * a.page) * token;
  };
  const int layer0 = blockIdx.y * a.layers_per_cta;
  const int layers = min(a.layers_per_cta, a.layers - layer0);
  for (int x = tid; x < layers * 2 * a.units; x += kMoveThreads) {
    const int y = a.by_units.of(x), layer = y >> 1, u = x - y * a.units;
    const int h = a.by_head.of(u);
    char* const base = ((y & 1) != 0 ? a.v : a.k) + (layer0 + layer) * a.layer + h * a.head +
                       static_cast<int64_t>(u - h * a.head_units) * sizeof(U);
    for (int m = 0; m < moves; m += 4) {
      U w[4];
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (m + e < moves) w[e] = *reinterpret_cast<const U*>(base + offset(from[list[m + e]], a.block, a.token));
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (m + e < moves) *reinterpret_cast<U*>(base + offset(to[list[m + e]], a.block, a.token)) = w[e];
    }
  }
  if (a.k_exps != nullptr)
    for (int x = tid; x < layers * 2 * a.kv_heads; x += kMoveThreads) {
      const int y = x / a.kv_heads, h = x - y * a.kv_heads;
      int8_t* const base = ((y & 1) != 0 ? a.v_exps : a.k_exps) + (layer0 + (y >> 1)) * a.e_layer + h * a.e_head;
      for (int m = 0; m < moves; ++m)
        base[offset(to[list[m]], a.e_block, a.e_token)] = base[offset(from[list[m]], a.e_block, a.e_token)];
    }
  if (err != 0 && blockIdx.y == 0 && a.dev_error != nullptr) atomicOr(a.dev_error, static_cast<int32_t>(err));
}

int padding_ctas(int n_rows) { return std::max(1, std::min(16, n_rows / 4096)); }
int tree_threads(int max_len) { return (max_len + 31) / 32 * 32; }

}  // namespace
}  // namespace serve
}  // namespace sv

extern "C" {

int spec_verify_tree(const int32_t* parents, const int32_t* seq_lens, const int32_t* row_offsets,
                     int32_t B, int32_t n_rows, int32_t max_len, int32_t* out_positions,
                     int32_t* out_mask, int32_t mask_words, int32_t* dev_error, void* stream) {
  using namespace sv::serve;
  if (B < 1 || n_rows < 0 || max_len < 1 || mask_words < (max_len + 31) / 32) return SV_ERR_ARG;
  if (max_len > SV_MAX_LEN || B > (1 << 24)) return SV_ERR_UNSUPPORTED;
  if (n_rows == 0) return SV_OK;  // an empty tensor has no address
  for (const void* p : {static_cast<const void*>(parents), static_cast<const void*>(seq_lens),
                        static_cast<const void*>(row_offsets), static_cast<const void*>(out_positions),
                        static_cast<const void*>(out_mask)})
    if (p == nullptr || !aligned_to(p, 4)) return SV_ERR_ARG;
  if (!null_or_aligned(dev_error, 4)) return SV_ERR_ARG;
  const PlanArgs a{parents, seq_lens, row_offsets, B, n_rows, max_len, mask_words,
                   out_positions, out_mask, dev_error};
  return launch(tree_plan_kernel, dim3(B + padding_ctas(n_rows)), tree_threads(max_len), 0, 1, false,
                static_cast<cudaStream_t>(stream), a);
}

int spec_verify_tree_accept(const int32_t* tokens, const int32_t* next_tokens,
                            const int32_t* parents, const int32_t* row_offsets, int32_t B,
                            int32_t n_rows, int32_t max_len, int32_t* out_tokens,
                            int32_t* out_path, int32_t* out_accept_len, int32_t* dev_error,
                            void* stream) {
  using namespace sv::serve;
  if (B < 1 || n_rows < 0 || max_len < 1) return SV_ERR_ARG;
  if (max_len > SV_MAX_LEN || B > (1 << 24)) return SV_ERR_UNSUPPORTED;
  for (const void* p : {static_cast<const void*>(row_offsets), static_cast<const void*>(out_accept_len)})
    if (p == nullptr || !aligned_to(p, 4)) return SV_ERR_ARG;
  for (const void* p : {static_cast<const void*>(tokens), static_cast<const void*>(next_tokens),
                        static_cast<const void*>(parents), static_cast<const void*>(out_tokens),
                        static_cast<const void*>(out_path)})
    if ((p == nullptr && n_rows > 0) || !aligned_to(p, 4)) return SV_ERR_ARG;
  if (!null_or_aligned(dev_error, 4)) return SV_ERR_ARG;
  const AcceptArgs a{tokens, next_tokens, parents, row_offsets, B, n_rows, max_len,
                     out_tokens, out_path, out_accept_len, dev_error};
  return launch(tree_accept_kernel, dim3(B + padding_ctas(n_rows)), tree_threads(max_len), 0, 1, false,
                static_cast<cudaStream_t>(stream), a);
}

int spec_verify_tree_move(const int32_t* path, const int32_t* accept_len,
                          const int32_t* row_offsets, const int64_t* slots, int32_t B,
                          int32_t n_rows, int32_t max_len, int32_t layers, int32_t kv_heads,
                          int32_t head_dim, void* key_cache, void* value_cache,
                          int64_t layer_stride, int64_t block_stride, int64_t token_stride,
                          int64_t head_stride, int32_t num_blocks, int32_t page_size,
                          int32_t cache_dtype, int8_t* key_exps, int8_t* value_exps,
                          int64_t e_layer_stride, int64_t e_block_stride, int64_t e_token_stride,
                          int64_t e_head_stride, int32_t* dev_error, void* stream) {
  using namespace sv::serve;
  if (cache_dtype != SV_BF16 && cache_dtype != SV_FP32 && cache_dtype != SV_E4M3) return SV_ERR_DTYPE;
  const int es = cache_dtype == SV_BF16 ? 2 : cache_dtype == SV_FP32 ? 4 : 1;
  if (B < 1 || n_rows < 0 || max_len < 1 || layers < 1 || kv_heads < 1 || head_dim < 1 ||
      num_blocks < 1 || page_size < 1)
    return SV_ERR_ARG;
  if (max_len > SV_MAX_LEN || B > (1 << 24) || static_cast<int64_t>(kv_heads) * head_dim > (1 << 20) ||
      layers > (1 << 14))
    return SV_ERR_UNSUPPORTED;
  for (int64_t s : {layer_stride, block_stride, token_stride, head_stride, e_layer_stride,
                    e_block_stride, e_token_stride, e_head_stride})
    if (s < 0) return SV_ERR_ARG;
  if (n_rows == 0) return SV_OK;  // an empty tensor has no address
  for (const void* p : {static_cast<const void*>(path), static_cast<const void*>(accept_len),
                        static_cast<const void*>(row_offsets)})
    if (p == nullptr || !aligned_to(p, 4)) return SV_ERR_ARG;
  if (slots == nullptr || !aligned_to(slots, 8) || key_cache == nullptr || value_cache == nullptr ||
      !null_or_aligned(dev_error, 4))
    return SV_ERR_ARG;
  if (cache_dtype == SV_E4M3 && (key_exps == nullptr || value_exps == nullptr)) return SV_ERR_ARG;
  if (cache_dtype != SV_E4M3) key_exps = value_exps = nullptr;
  uint64_t mix = reinterpret_cast<uint64_t>(key_cache) | reinterpret_cast<uint64_t>(value_cache);
  // a dimension of one is never stepped along, whatever its stride says
  for (int64_t s : {layers > 1 ? layer_stride : 0, num_blocks > 1 ? block_stride : 0,
                    page_size > 1 ? token_stride : 0, kv_heads > 1 ? head_stride : 0,
                    static_cast<int64_t>(head_dim)})
    mix |= static_cast<uint64_t>(s) * es;
  if (mix % es != 0) return SV_ERR_ARG;
  const int unit = mix % 16 == 0 ? 16 : mix % 8 == 0 ? 8 : mix % 4 == 0 ? 4 : mix % 2 == 0 ? 2 : 1;
  Device d;
  const int rc = device(&d);
  if (rc != SV_OK) return rc;
  const int units = kv_heads * head_dim * es / unit;
  // layers a CTA: all, until there are some CTAs for every SM
  const int parts = std::min(layers, std::max(1, (4 * d.sms + B - 1) / B));
  const int per = (layers + parts - 1) / parts;
  MoveArgs a{path, accept_len, row_offsets, slots, B, n_rows, max_len, layers, per,
             static_cast<char*>(key_cache), static_cast<char*>(value_cache), layer_stride * es,
             block_stride * es, token_stride * es, head_stride * es, key_exps, value_exps,
             e_layer_stride, e_block_stride, e_token_stride, e_head_stride,
             static_cast<int64_t>(num_blocks) * page_size, page_size, kv_heads, units,
             head_dim * es / unit, dev_error,
             FastDiv::by(static_cast<uint32_t>(head_dim * es / unit)),
             FastDiv::by(static_cast<uint32_t>(units))};
  if (static_cast<int64_t>(per) * 2 * units > INT32_MAX) return SV_ERR_UNSUPPORTED;
  const dim3 grid(static_cast<unsigned>(B), static_cast<unsigned>((layers + per - 1) / per));
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  switch (unit) {
    case 16: return launch(tree_move_kernel<uint4>, grid, kMoveThreads, 0, 1, false, st, a);
    case 8: return launch(tree_move_kernel<uint2>, grid, kMoveThreads, 0, 1, false, st, a);
    case 4: return launch(tree_move_kernel<uint32_t>, grid, kMoveThreads, 0, 1, false, st, a);
    case 2: return launch(tree_move_kernel<uint16_t>, grid, kMoveThreads, 0, 1, false, st, a);
    default: return launch(tree_move_kernel<uint8_t>, grid, kMoveThreads, 0, 1, false, st, a);
  }
}

}  // extern "C"
