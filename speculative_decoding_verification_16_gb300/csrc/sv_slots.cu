// sv_slots.cu -- block tables, slot maps and cache writes of a paged server
// (include/spec_verify_serve.h).
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <mutex>

#include "sv_host.cuh"

namespace sv {
namespace serve {

namespace {
constexpr int kMaxDevices = 64;
std::mutex g_mu;
Device g_dev[kMaxDevices];
struct Allowed {
  int dev;
  const void* fn;
};
constexpr int kMaxAllowed = 256;
Allowed g_allowed[kMaxAllowed];
int g_nallowed = 0;
}  // namespace

int device(Device* out) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return SV_ERR_CUDA;
  std::lock_guard<std::mutex> lock(g_mu);
  Device& d = g_dev[dev];
  if (d.sms == 0) {
    Device n;
    if (cudaDeviceGetAttribute(&n.sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&n.max_smem, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev) !=
            cudaSuccess)
      return SV_ERR_CUDA;
    d = n;
  }
  *out = d;
  return SV_OK;
}

int allow_smem(const void* kernel, int max_smem) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return SV_ERR_CUDA;
  std::lock_guard<std::mutex> lock(g_mu);
  for (int i = 0; i < g_nallowed; ++i)
    if (g_allowed[i].dev == dev && g_allowed[i].fn == kernel) return SV_OK;
  cudaFuncAttributes fa{};
  if (cudaFuncGetAttributes(&fa, kernel) != cudaSuccess ||
      cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           max_smem - static_cast<int>(fa.sharedSizeBytes)) != cudaSuccess)
    return SV_ERR_CUDA;
  if (g_nallowed < kMaxAllowed) g_allowed[g_nallowed++] = Allowed{dev, kernel};
  return SV_OK;
}

// ---------------------------------------------------------------- slots
//
// Three prefix sums over the requests (new tokens, pages given back, pages
// taken) decide everything: the k-th page taken in the call is the k-th from
// the top of the free list after the returns, so any thread finds any page id
// by itself and no CTA waits for another.  Every CTA forms the sums over all
// requests (12 bytes each, from L2) and then does its share of the tokens,
// table entries and returned pages.  What a CTA reads no CTA writes: table
// entries below `held`, list entries below `free_count`.
//
// Latency bound: the launch, two dependent rounds of loads (lengths, then page
// ids) and the block scan between them: 5.2 us for 32 requests of 16 tokens, 9.0 us
// for 1,024 requests and 131,000 tokens, whose 1.6 MB take 0.24 us at the copy rate.
constexpr int kSlotThreads = 512;
constexpr int kSlotWarps = kSlotThreads / 32;
constexpr int kSlotRowsPerCta = 1024;

struct SlotsArgs {
  const int32_t *ctx, *fresh;
  int32_t B, page;
  int32_t* table;
  int64_t table_stride;
  int32_t width;
  const int32_t* held;
  int32_t* free_list;
  int32_t free_cap;
  const int32_t* free_count;
  int32_t n_rows;
  int32_t *row_offsets, *seq_lens, *positions;
  int64_t* slots;
  int32_t *held_out, *free_count_out, *dev_error;
  FastDiv by_page;
};

struct Request {
  int32_t ctx, fresh, held, need;
  bool ok;  // lengths and counts in range: takes part in the page exchange
};

__device__ __forceinline__ Request load_request(const SlotsArgs& a, int r) {
  Request q;
  q.ctx = a.ctx[r];
  q.fresh = a.fresh[r];
  q.held = a.held[r];
  const bool rows_ok = q.fresh >= 0 && q.fresh <= a.n_rows;
  if (!rows_ok) q.fresh = 0;
  const uint32_t seq = static_cast<uint32_t>(q.ctx) + static_cast<uint32_t>(q.fresh);
  q.ok = rows_ok && q.ctx >= 0 && seq <= INT32_MAX && q.held >= 0 && q.held <= a.width;
  q.need = q.held;
  if (q.ok) {
    const int pages = a.by_page.of(static_cast<int>(seq));
    const int need = pages + (static_cast<int>(seq) > pages * a.page ? 1 : 0);
    if (need <= a.width) q.need = need;
    else q.ok = false;
  }
  return q;
}

// Largest i in [0, n) with a[i] <= v; a rises and a[0] <= v.
template <typename T>
__device__ __forceinline__ int last_at_or_below(const T* a, int n, T v) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (a[mid] <= v) lo = mid; else hi = mid;
  }
  return lo;
}

__global__ __launch_bounds__(kSlotThreads) void slots_kernel(const SlotsArgs a) {
  extern __shared__ int32_t sm[];
  int32_t* offs = sm;              // [B + 1] rows before request r
  int32_t* give = offs + a.B + 1;  // [B + 1] pages given back before r
  int32_t* take = give + a.B + 1;  // [B + 1] pages taken before r
  int32_t* ctxs = take + a.B + 1;  // [B] context
  int32_t* keep = ctxs + a.B;      // [B] pages held before the call, -1: left out
  __shared__ int64_t part0[kSlotWarps];
  __shared__ int32_t part1[kSlotWarps], part2[kSlotWarps];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const bool first = blockIdx.x == 0;
  const int32_t cap_count = *a.free_count;
  const int32_t count = min(max(cap_count, 0), a.free_cap);
  uint32_t err = 0;

  int64_t c0 = 0;  // carried over the chunks
  int32_t c1 = 0, c2 = 0;
  for (int base = 0; base < a.B; base += kSlotThreads) {
    const int r = base + tid;
    int64_t s0 = 0;
    int32_t s1 = 0, s2 = 0;
    if (r < a.B) {
      const Request q = load_request(a, r);
      s0 = q.fresh;
      s1 = max(q.held - q.need, 0);
      s2 = max(q.need - q.held, 0);
      if (!q.ok) err |= SV_DEVERR_LEN;
      ctxs[r] = q.ctx, keep[r] = q.ok ? q.held : -1;
      // -1: attention leaves the request out; its table does not hold its tokens' pages
      if (first) a.seq_lens[r] = q.ok ? q.ctx + q.fresh : -1;
    }
    const int64_t own0 = s0;
    const int32_t own1 = s1, own2 = s2;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int64_t t0 = __shfl_up_sync(~0u, s0, d);
      const int32_t t1 = __shfl_up_sync(~0u, s1, d), t2 = __shfl_up_sync(~0u, s2, d);
      if (lane >= d) s0 += t0, s1 += t1, s2 += t2;
    }
    if (lane == 31) part0[warp] = s0, part1[warp] = s1, part2[warp] = s2;
    __syncthreads();
    int64_t p0 = c0;
    int32_t p1 = c1, p2 = c2;
    for (int w = 0; w < kSlotWarps; ++w) {
      if (w < warp) p0 += part0[w], p1 += part1[w], p2 += part2[w];
      c0 += part0[w], c1 += part1[w], c2 += part2[w];
    }
    if (r < a.B) {  // row sums stop at 2^31 - 1: what lies past n_rows is not used
      offs[r] = static_cast<int32_t>(min(p0 + s0 - own0, static_cast<int64_t>(INT32_MAX)));
      give[r] = p1 + s1 - own1;
      take[r] = p2 + s2 - own2;
    }
    __syncthreads();
  }
  if (tid == 0) {
    offs[a.B] = static_cast<int32_t>(min(c0, static_cast<int64_t>(INT32_MAX)));
    give[a.B] = c1, take[a.B] = c2;
  }
  __syncthreads();
  const int32_t returned = c1;
  const int64_t avail = static_cast<int64_t>(count) + returned;

  // the i-th page given back in this call
  auto returned_page = [&](int32_t i) {
    const int r = last_at_or_below(give, a.B, i);
    const int32_t need = keep[r] - (give[r + 1] - give[r]);
    return a.table[r * a.table_stride + need + (i - give[r])];
  };
  // the k-th page taken: k-th from the top of the list after the returns
  auto taken_page = [&](int32_t k) {
    const int64_t i = avail - 1 - k;
    return i < count ? a.free_list[i] : returned_page(static_cast<int32_t>(i - count));
  };

  if (first) {
    for (int r = tid; r <= a.B; r += kSlotThreads) a.row_offsets[r] = offs[r];
    for (int r = tid; r < a.B; r += kSlotThreads) {
      const int32_t taken = take[r + 1] - take[r];
      const bool served = take[r + 1] <= avail || taken == 0;
      if (!served) err |= SV_DEVERR_BLOCKS, a.seq_lens[r] = -1;  // over this thread's own store
      a.held_out[r] = keep[r] < 0 ? a.held[r]
                                  : keep[r] + (served ? taken : 0) - (give[r + 1] - give[r]);
    }
    if (tid == 0) {
      const int r = last_at_or_below(take, a.B + 1, static_cast<int32_t>(
          min(avail, static_cast<int64_t>(INT32_MAX))));
      *a.free_count_out = static_cast<int32_t>(avail - take[r]);
      if (cap_count != count || avail > a.free_cap || offs[a.B] > a.n_rows) err |= SV_DEVERR_LEN;
    }
  }
  const int64_t step = static_cast<int64_t>(gridDim.x) * kSlotThreads;
  const int64_t start = static_cast<int64_t>(blockIdx.x) * kSlotThreads + tid;
  for (int64_t i = start; i < returned; i += step)
    if (count + i < a.free_cap) a.free_list[count + i] = returned_page(static_cast<int32_t>(i));
  for (int64_t k = start; k < take[a.B]; k += step) {
    const int r = last_at_or_below(take, a.B, static_cast<int32_t>(k));
    if (take[r + 1] > avail) continue;  // not served
    a.table[r * a.table_stride + keep[r] + (k - take[r])] =
        taken_page(static_cast<int32_t>(k));
  }
  for (int64_t i = start; i < a.n_rows; i += step) {
    int32_t pos = 0;
    int64_t slot = -1;
    if (i < offs[a.B]) {
      const int r = last_at_or_below(offs, a.B, static_cast<int32_t>(i));
      if (keep[r] >= 0) {
        pos = ctxs[r] + static_cast<int32_t>(i) - offs[r];
        const int32_t col = a.by_page.of(pos);
        int32_t id = -1;
        if (col < keep[r])
          id = a.table[r * a.table_stride + col];
        else if (take[r + 1] <= avail)
          id = taken_page(take[r] + col - keep[r]);
        if (id >= 0) slot = static_cast<int64_t>(id) * a.page + (pos - col * a.page);
      }
    }
    a.positions[i] = pos;
    a.slots[i] = slot;
  }
  if (err != 0 && a.dev_error != nullptr) atomicOr(a.dev_error, static_cast<int32_t>(err));
}

// ---------------------------------------------------------------- append
//
// A copy of rows to scattered places: U-byte units, one CTA a group of R rows,
// a thread the same unit of each row of the group, so that its R loads are in
// flight together.  HBM bound: every byte read and written once.  16,384 rows of
// 8 x 128 bf16 (134 MB) 25.5 us, 5.3 TB/s, 0.79 of the measured copy rate; 512 rows
// 2.8 us, of which the launch is most.
constexpr int kAppendThreads = 256;

struct AppendArgs {
  const char *key, *value;
  int64_t k_row, k_head, v_row, v_head;  // bytes
  const int64_t* slots;
  int32_t n_rows, units, head_units;  // units per row, per head
  char *k_cache, *v_cache;
  int64_t block, token, head;  // bytes
  int64_t n_slots;
  int32_t page;
  int32_t* dev_error;
};

template <typename U, int R>
__global__ __launch_bounds__(kAppendThreads) void append_kernel(const AppendArgs a) {
  const int64_t row0 = static_cast<int64_t>(blockIdx.x) * R;
  int64_t at[R];  // byte offset of the row's token in the caches, or -1
  uint32_t err = 0;
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const int64_t row = row0 + i;
    const int64_t slot = row < a.n_rows ? a.slots[row] : -1;
    if (slot >= a.n_slots) err = SV_DEVERR_PAGE;
    if (slot < 0 || slot >= a.n_slots) {
      at[i] = -1;
    } else {
      const int64_t b = slot / a.page;
      at[i] = b * a.block + (slot - b * a.page) * a.token;
    }
  }
  for (int v = threadIdx.x; v < 2 * a.units; v += kAppendThreads) {
    const bool val = v >= a.units;
    const int u = val ? v - a.units : v;
    const int h = u / a.head_units;
    const int64_t in_head = static_cast<int64_t>(u - h * a.head_units) * sizeof(U);
    const char* src = (val ? a.value : a.key) + h * (val ? a.v_head : a.k_head) + in_head;
    const int64_t src_row = val ? a.v_row : a.k_row;
    char* dst = (val ? a.v_cache : a.k_cache) + h * a.head + in_head;
    U x[R];
#pragma unroll
    for (int i = 0; i < R; ++i)
      if (at[i] >= 0) x[i] = *reinterpret_cast<const U*>(src + (row0 + i) * src_row);
#pragma unroll
    for (int i = 0; i < R; ++i)
      if (at[i] >= 0) *reinterpret_cast<U*>(dst + at[i]) = x[i];
  }
  if (err != 0 && threadIdx.x == 0 && a.dev_error != nullptr)
    atomicOr(a.dev_error, static_cast<int32_t>(err));
}

template <typename U>
int launch_append(const AppendArgs& a, cudaStream_t st) {
  // a few rows: one a CTA, to spread them; more: four loads in flight a thread
  if (a.n_rows <= 304)
    return launch(append_kernel<U, 1>, dim3(a.n_rows), kAppendThreads, 0, 1, false, st, a);
  return launch(append_kernel<U, 4>, dim3((a.n_rows + 3) / 4), kAppendThreads, 0, 1, false, st, a);
}

}  // namespace serve
}  // namespace sv

extern "C" {

int spec_verify_slots(const int32_t* context_lens, const int32_t* verify_lens, int32_t B,
                      int32_t page_size, int32_t* block_table, int64_t table_stride,
                      int32_t width, const int32_t* held, int32_t* free_list, int32_t free_cap,
                      const int32_t* free_count, int32_t n_rows, int32_t* out_row_offsets,
                      int32_t* out_seq_lens, int32_t* out_positions, int64_t* out_slots,
                      int32_t* out_held, int32_t* out_free_count, int32_t* dev_error,
                      void* stream) {
  using sv::serve::aligned_to;
  if (B < 1 || page_size < 1 || width < 1 || table_stride < width || free_cap < 0 || n_rows < 0)
    return SV_ERR_ARG;
  if (static_cast<int64_t>(B) * width > INT32_MAX) return SV_ERR_UNSUPPORTED;
  if (B > SV_SLOTS_MAX_B) return SV_ERR_UNSUPPORTED;
  for (const void* p : {static_cast<const void*>(context_lens),
                        static_cast<const void*>(verify_lens), static_cast<const void*>(held),
                        static_cast<const void*>(free_count),
                        static_cast<const void*>(block_table),
                        static_cast<const void*>(out_row_offsets),
                        static_cast<const void*>(out_seq_lens),
                        static_cast<const void*>(out_held),
                        static_cast<const void*>(out_free_count)})
    if (p == nullptr || !aligned_to(p, 4)) return SV_ERR_ARG;
  if ((free_cap > 0 && free_list == nullptr) || !aligned_to(free_list, 4) ||
      !sv::serve::null_or_aligned(dev_error, 4))
    return SV_ERR_ARG;
  if (n_rows > 0 && (out_positions == nullptr || out_slots == nullptr)) return SV_ERR_ARG;
  if (!aligned_to(out_positions, 4) || !aligned_to(out_slots, 8)) return SV_ERR_ARG;
  // CTAs read these while others write the results
  const struct {
    const void* at;
    int64_t bytes;
  } in[] = {{context_lens, 4 * int64_t{B}}, {verify_lens, 4 * int64_t{B}},
            {held, 4 * int64_t{B}}, {free_count, 4}},
    results[] = {{out_row_offsets, 4 * (int64_t{B} + 1)}, {out_seq_lens, 4 * int64_t{B}},
                 {out_positions, 4 * int64_t{n_rows}}, {out_slots, 8 * int64_t{n_rows}},
                 {out_held, 4 * int64_t{B}}, {out_free_count, 4}};
  for (const auto& o : results)
    for (const auto& i : in)
      if (o.bytes > 0 && static_cast<const char*>(o.at) < static_cast<const char*>(i.at) + i.bytes &&
          static_cast<const char*>(i.at) < static_cast<const char*>(o.at) + o.bytes)
        return SV_ERR_ARG;
  sv::serve::Device d;
  const int rc = sv::serve::device(&d);
  if (rc != SV_OK) return rc;
  const sv::serve::SlotsArgs a{context_lens, verify_lens, B, page_size, block_table, table_stride,
                               width, held, free_list, free_cap, free_count, n_rows,
                               out_row_offsets, out_seq_lens, out_positions, out_slots, out_held,
                               out_free_count, dev_error,
                               sv::serve::FastDiv::by(static_cast<uint32_t>(page_size))};
  const int grid = std::max(1, std::min(d.sms, (n_rows + sv::serve::kSlotRowsPerCta - 1) /
                                                   sv::serve::kSlotRowsPerCta));
  return sv::serve::launch(sv::serve::slots_kernel, dim3(grid), sv::serve::kSlotThreads,
                           (5 * B + 3) * 4, 1, false, static_cast<cudaStream_t>(stream), a);
}

int spec_verify_append(const void* key, const void* value, int64_t k_row_stride,
                       int64_t k_head_stride, int64_t v_row_stride, int64_t v_head_stride,
                       const int64_t* slots, int32_t n_rows, int32_t kv_heads, int32_t head_dim,
                       void* key_cache, void* value_cache, int64_t block_stride,
                       int64_t token_stride, int64_t head_stride, int32_t num_blocks,
                       int32_t page_size, int32_t dtype, int32_t* dev_error, void* stream) {
  using namespace sv::serve;
  if (dtype != SV_BF16 && dtype != SV_FP32) return SV_ERR_DTYPE;
  const int es = dtype == SV_BF16 ? 2 : 4;
  if (n_rows < 0 || kv_heads < 1 || head_dim < 1 || num_blocks < 1 || page_size < 1)
    return SV_ERR_ARG;
  if (k_row_stride < 0 || k_head_stride < 0 || v_row_stride < 0 || v_head_stride < 0 ||
      block_stride < 0 || token_stride < 0 || head_stride < 0)
    return SV_ERR_ARG;
  if (n_rows == 0) return SV_OK;
  if (key == nullptr || value == nullptr || slots == nullptr || key_cache == nullptr ||
      value_cache == nullptr || !aligned_to(slots, 8) || !null_or_aligned(dev_error, 4))
    return SV_ERR_ARG;
  if (static_cast<int64_t>(kv_heads) * head_dim > (1 << 24)) return SV_ERR_UNSUPPORTED;
  // the widest unit that every address is a multiple of
  uint64_t mix = reinterpret_cast<uint64_t>(key) | reinterpret_cast<uint64_t>(value) |
                 reinterpret_cast<uint64_t>(key_cache) | reinterpret_cast<uint64_t>(value_cache);
  for (int64_t s : {k_row_stride, k_head_stride, v_row_stride, v_head_stride, block_stride,
                    token_stride, head_stride, static_cast<int64_t>(head_dim)})
    mix |= static_cast<uint64_t>(s) * es;
  if (mix % es != 0) return SV_ERR_ARG;
  const int unit = mix % 16 == 0 ? 16 : mix % 8 == 0 ? 8 : mix % 4 == 0 ? 4 : 2;
  AppendArgs a{static_cast<const char*>(key), static_cast<const char*>(value),
               k_row_stride * es, k_head_stride * es, v_row_stride * es, v_head_stride * es,
               slots, n_rows, kv_heads * head_dim * es / unit, head_dim * es / unit,
               static_cast<char*>(key_cache), static_cast<char*>(value_cache),
               block_stride * es, token_stride * es, head_stride * es,
               static_cast<int64_t>(num_blocks) * page_size, page_size, dev_error};
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  switch (unit) {
    case 16: return launch_append<uint4>(a, st);
    case 8: return launch_append<uint2>(a, st);
    case 4: return launch_append<uint32_t>(a, st);
    default: return launch_append<uint16_t>(a, st);
  }
}

}  // extern "C"
