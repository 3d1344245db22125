// sv_attn_mma.cuh -- the tensor core attention kernel (bf16).
//
// The query rows of a request that share a key/value head -- l tokens times the
// group of G heads -- are packed into tiles of 128 rows, row i = token i / G,
// head i % G of the group, so a key/value tile is read once for all of them.
// An item is (request, kv head, NS row tiles); its work is the 64-key tiles
// from the first key that its first row sees to the last that its last row
// sees.  All items' tiles in a row are cut into equal runs, one a worker (CTA);
// a worker whose run starts or ends inside an item leaves an unnormalised
// partial (O, m, l) in the workspace, and the combine kernel joins them.
//
// Per stream of 128 rows (one softmax warpgroup, a thread a row) and key tile:
//   S = Q K^T   tcgen05.mma from shared memory into 64 tensor memory columns
//   P = 2^(S c - m c), c = scale log2 e, rounded to bf16 over S's own columns
//   O += P V    tcgen05.mma with P from tensor memory
// S has two buffers, and Q K^T runs two tiles ahead of P V, so that neither the
// softmax nor the tensor core waits for the other's latency.  (128-key tiles
// with one buffer: 3,400 cycles from S to P beside 1,024 of products a stream
// and tile, 1.58 ms for the 4,096-token chunks; two warpgroups a stream to halve
// the softmax: 1.77 ms.)  The running maximum m of a row rises lazily: P may grow
// to 2^8 before O is rescaled, so most tiles leave O alone; the row sum l is of
// the unrounded P, in fp32.  P keeps 8 significant bits: an error of at most 2^-8
// a weight, of the size of the output's own rounding, for tensor products at
// full rate.
//
// NS = 1 (at most 128 rows an item, decoding and verify steps: the cache's
// bytes bound it): two CTAs an SM, each with one stream; for heads above 128, whose
// O fills half the tensor memory, one CTA an SM at any number of rows.
// NS = 2 (longer chunks: the products bound it): one CTA an SM, two streams
// over the same key/value tiles, the tensor core alternating between them.  At head_dim
// 128 a stream's tile takes 8 x 48 + 4 x 64 = 640 cycles of the tensor core, Q K^T being
// bound by reading both operands from shared memory, for 512 of arithmetic: no more
// than 0.80 of the rate, of which 0.69 is reached.  One call has one NS, by max_len: single
// tokens beside a chunk run with one of two streams idle (200 over 4,096 keys 500 us
// alone, 722 with one chunk of 512 that alone takes 38).
//
// Keys and values come by tensor copies of whole page pieces (page sizes that
// are a multiple of 64 or 8, 16, 32) and by 16-byte copies of single rows
// otherwise.
//
// Masked places.  S of a masked key is replaced, whatever it holds.  A masked
// value is multiplied by P = 0, so a NaN or infinity there would reach every
// row: in the tiles that not all rows see whole, V's non-finite elements under
// keys that some row does not see are set to 0 in shared memory, and the
// epilogue adds them, from the cache, to the rows that do see them.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>

#include "sv_ptx.cuh"
#include "sv_tcgen05.cuh"

namespace sv {
namespace serve {

constexpr int kRows = 128;        // query rows of a stream
constexpr int kTile = 64;         // keys of a tile
constexpr int kMaxWorkers = 320;  // most CTAs of heads up to 128 with one stream
constexpr int kMinRun = 3;        // least tiles of a worker's run
constexpr float kRescale = 8.0f;  // log2 of how far P may exceed 1 before O is rescaled

struct AttnRecord {  // of a worker whose run is the second in an item
  int32_t parts;  // runs that the item is cut into; 0 for another worker
  int32_t rows, row0, h, m;  // the item's rows, its request's first row, head and row tile
};

struct MmaArgs {
  AttnArgs a;
  int32_t kv_heads, box;  // box: tokens of a tensor copy; 0: copies of single rows
  bool whole;             // items are not cut
  AttnRecord* record;     // [kMaxWorkers]
  float2* ml;             // [2 * kMaxWorkers][rows]: m c and l of the partials
  float4* o;              // [2 * kMaxWorkers][DP / 4][rows]
};

constexpr int kMaxUnits = 10;
__host__ __device__ constexpr int attn_units(int ns, int dp) { return ns == 1 && dp >= 128 ? 5 : kMaxUnits; }
// CTAs an SM.
__host__ __device__ constexpr int attn_per_sm(int ns, int dp) { return ns == 1 && dp <= 128 ? 2 : 1; }
__host__ __device__ constexpr int attn_threads(int ns) { return ns * 6 * 32; }  // softmax, copies, products
// query tiles, ring of key and value tiles, barriers, the softmax warps' walks
__host__ __device__ constexpr int attn_smem(int ns, int dp) {
  return ns * kRows * dp * 2 + attn_units(ns, dp) * kTile * dp * 2 + 320 + ns * 4 * 104;
}

// ---------------------------------------------------------------- work
struct Segment {  // consecutive tiles of one item
  int r, h, m;
  int row0, l, seq;
  int tile0, tile1;   // key tiles [tile0, tile1)
  int rows;           // valid rows of the item
  int kv_end;         // keys past the last one that any row sees
  bool begins, whole;
};

struct ItemTiles {
  int lo, tiles, rows, kv_end;
  int n;  // its share of the work: the tiles, or 1 where items are not cut
};

template <int MR>
__device__ __forceinline__ ItemTiles item_tiles(const MmaArgs& p, const Span& s, int m) {
  const AttnArgs& a = p.a;
  ItemTiles t;
  const int all = s.l * a.group;
  t.rows = min(MR, all - m * MR);
  const int j0 = a.by_group.of(m * MR), j1 = a.by_group.of(m * MR + t.rows - 1);
  t.kv_end = max(0, s.seq - s.l + j1 + 1);
  const int kv_lo = a.window > 0 ? max(0, s.seq - s.l + j0 - a.window + 1) : 0;
  t.lo = kv_lo / kTile;
  t.tiles = max(1, (t.kv_end + kTile - 1) / kTile - t.lo);
  t.n = p.whole ? 1 : t.tiles;
  return t;
}

template <int MR>
__device__ __forceinline__ int64_t head_tiles(const MmaArgs& p, const Span& s) {
  int64_t n = 0;
  if (s.l > 0)
    for (int m = 0; m * MR < s.l * p.a.group; ++m) n += item_tiles<MR>(p, s, m).n;
  return n;
}

// Products with up to kMaxWorkers fit 32 bits below this total: 64-bit division
// takes hundreds of cycles.
constexpr int64_t kSmallTotal = int64_t{1} << 22;
__device__ __forceinline__ int64_t worker_start(int64_t total, int workers, int w) {
  if (total < kSmallTotal) return static_cast<uint32_t>(total) * w / static_cast<uint32_t>(workers);
  return total * w / workers;
}
__device__ __forceinline__ int worker_of(int64_t total, int workers, int64_t u) {
  if (total < kSmallTotal)
    return static_cast<int>((static_cast<uint32_t>(u + 1) * workers - 1) / static_cast<uint32_t>(total));
  return static_cast<int>(((u + 1) * workers - 1) / total);
}

template <int MR>
struct Walk {  // a worker's segments in order
  int r, h, m, off;
  int64_t left;
  Span s;

  __device__ __forceinline__ bool next(const MmaArgs& p, Segment* g) {
    if (left <= 0) return false;
    const ItemTiles t = item_tiles<MR>(p, s, m);
    const int take = static_cast<int>(min(left, static_cast<int64_t>(t.n - off)));
    g->r = r, g->h = h, g->m = m, g->row0 = s.row0, g->l = s.l, g->seq = s.seq;
    g->tile0 = t.lo + off, g->tile1 = t.lo + (p.whole ? t.tiles : off + take);
    g->rows = t.rows, g->kv_end = t.kv_end;
    g->begins = off == 0, g->whole = off == 0 && take == t.n;
    left -= take;
    off += take;
    if (off == t.n) {
      off = 0;
      if (++m * MR >= s.l * p.a.group) {
        m = 0;
        if (++h == p.kv_heads) {
          h = 0;
          if (left > 0) do s = span_of(p.a, ++r); while (s.l <= 0);
        }
      }
    }
    return true;
  }
};

template <int MR>
struct PlanSmem {
  int64_t part[16];
  Walk<MR> walk;
};

// Every CTA finds its own run from the requests' lengths: a scan over the
// requests' tiles, then the thread whose request holds the run's start sets out
// the walk.  More requests than threads: the tiles are formed twice, once for the
// total and once up to the start.
template <int MR, int THREADS>
__device__ __forceinline__ bool plan(const MmaArgs& p, PlanSmem<MR>* sm, Walk<MR>* w) {
  const AttnArgs& a = p.a;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  constexpr int kW = THREADS / 32;
  Span s{0, 0, 0};
  int64_t mine = 0, per_head = 0;
  bool bad = false;
  for (int r = tid; r < a.B; r += THREADS) {
    s = span_of(a, r, &bad);
    per_head = head_tiles<MR>(p, s);
    mine += per_head;
  }
  if (bad && blockIdx.x == 0 && a.dev_error != nullptr) atomicOr(a.dev_error, SV_DEVERR_LEN);
  mine *= p.kv_heads;
  int64_t inc = mine;  // up to and with this thread's requests
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int64_t o = __shfl_up_sync(~0u, inc, d);
    if (lane >= d) inc += o;
  }
  if (lane == 31) sm->part[warp] = inc;
  __syncthreads();
  int64_t total = 0, before = inc - mine;
#pragma unroll
  for (int i = 0; i < kW; ++i) {
    if (i < warp) before += sm->part[i];
    total += sm->part[i];
  }
  // runs of at least three tiles: shorter ones cost more in partials and their join
  // than they save (one request's verify step 17.8 us at one, 15.7 at three, 18.2 at
  // four; 8 requests of 16 tokens over up to 2,000 keys 22.1, 22.2, 21.2)
  const int workers = static_cast<int>(
      min(static_cast<int64_t>(gridDim.x), p.whole ? total : (total + kMinRun - 1) / kMinRun));
  const int me = blockIdx.x;
  if (me >= workers) {
    if (tid == 0) p.record[me] = AttnRecord{0, 0, 0, 0, 0};
    return false;
  }
  const int64_t start = worker_start(total, workers, me);
  // by the thread with request r, `rem` tiles into it
  int item = -1;  // its item's tiles, in that thread
  auto set_out = [&](int r, int64_t rem) {
    Walk<MR> x;
    x.r = r, x.s = s;
    x.h = rem < (1 << 30) && per_head < (1 << 30)
              ? static_cast<int>(static_cast<uint32_t>(rem) / static_cast<uint32_t>(per_head))
              : static_cast<int>(rem / per_head);
    rem -= x.h * per_head;
    x.m = 0;
    ItemTiles t = item_tiles<MR>(p, s, 0);
    while (rem >= t.n) rem -= t.n, t = item_tiles<MR>(p, s, ++x.m);
    x.off = static_cast<int>(rem);
    x.left = worker_start(total, workers, me + 1) - start;
    sm->walk = x;
    item = t.n;
  };
  if (a.B <= THREADS) {
    if (before <= start && start < before + mine) set_out(tid, start - before);
  } else {
    int64_t carry = 0;
    for (int base = 0; base < a.B && carry <= start; base += THREADS) {
      const int r = base + tid;
      s = r < a.B ? span_of(a, r) : Span{0, 0, 0};
      per_head = head_tiles<MR>(p, s);
      mine = per_head * p.kv_heads;
      inc = mine;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int64_t o = __shfl_up_sync(~0u, inc, d);
        if (lane >= d) inc += o;
      }
      __syncthreads();
      if (lane == 31) sm->part[warp] = inc;
      __syncthreads();
      before = carry + inc - mine;
#pragma unroll
      for (int i = 0; i < kW; ++i) {
        if (i < warp) before += sm->part[i];
        carry += sm->part[i];
      }
      if (before <= start && start < before + mine) set_out(r, start - before);
    }
  }
  __syncthreads();
  *w = sm->walk;
  if (item >= 0) {  // the record, while the others go on
    AttnRecord rec{0, 0, 0, 0, 0};
    const int64_t first = start - w->off;  // the item's first tile
    if (w->off > 0 && worker_of(total, workers, first) == me - 1)
      rec = AttnRecord{worker_of(total, workers, first + item - 1) - me + 2,
                       item_tiles<MR>(p, w->s, w->m).rows, w->s.row0, w->h, w->m};
    p.record[me] = rec;
  }
  return true;
}

// ---------------------------------------------------------------- kernel
template <int NS, int DP>
struct AttnSmem {
  static constexpr int kUnits = attn_units(NS, DP);
  static constexpr int kUnitBytes = kTile * DP * 2;
  static constexpr int kQBytes = kRows * DP * 2;
  static constexpr int kChunks = DP / 64;
};

struct AttnBars {
  uint64_t full[kMaxUnits], empty[kMaxUnits];
  uint64_t q[2], s[2][2], p[2][2], o[2][2], idle;  // by stream; s, p and o by S buffer too
  uint32_t tmem;
  int32_t odd;  // a non-finite value was set aside in this CTA
};
static_assert(sizeof(AttnBars) <= 320, "barrier block");

// The ring's order in a segment of n tiles is that of the products: K 0, K 1,
// V 0, K 2, V 1, K 3, ..  Positions of the K and the V of tile i:
__device__ __forceinline__ int k_position(int i) { return i < 2 ? i : 2 * i - 1; }
__device__ __forceinline__ int v_position(int n, int i) { return min(n, i + 2) + i; }

// Two floats at once: a * b + c and a + b.
__device__ __forceinline__ uint64_t pack2(float lo, float hi) {
  uint64_t v;
  asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(lo), "f"(hi));
  return v;
}
__device__ __forceinline__ void unpack2(uint64_t v, float* lo, float* hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(*lo), "=f"(*hi) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

template <int MR>
struct WarpWalk {
  Walk<MR> walk;
  Segment next;
};

template <int NS, int DP, bool TMA>
__global__ __launch_bounds__(attn_threads(NS), attn_per_sm(NS, DP)) void attn_mma_kernel(
    const MmaArgs p, const __grid_constant__ CUtensorMap kmap,
    const __grid_constant__ CUtensorMap vmap) {
  using L = AttnSmem<NS, DP>;
  constexpr int MR = NS * kRows;
  constexpr int kThreads = attn_threads(NS);
  constexpr uint32_t kCols = attn_per_sm(NS, DP) == 2 ? 256 : 512;
  // tensor memory columns: two S buffers of each stream, then O of each
  constexpr uint32_t kO = NS * 2 * kTile;
  extern __shared__ __align__(1024) char smem[];
  const AttnArgs& a = p.a;
  char* const qbuf = smem;
  char* const ring = smem + NS * L::kQBytes;
  AttnBars* const bars = reinterpret_cast<AttnBars*>(ring + L::kUnits * L::kUnitBytes);
  WarpWalk<MR>* const walks = reinterpret_cast<WarpWalk<MR>*>(reinterpret_cast<char*>(bars) + 320);
  static_assert(sizeof(WarpWalk<MR>) <= 104, "walk block");
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  constexpr int kSoftmax = NS * 4, kLoadWarp = kSoftmax, kMmaWarp = kSoftmax + NS;
  bool timed_out = false;

  if (tid == 0) {
    for (int i = 0; i < L::kUnits; ++i) {
      mbar_init(smem_addr(&bars->full[i]), TMA ? 1 : 32);
      mbar_init(smem_addr(&bars->empty[i]), NS);
    }
    for (int s = 0; s < NS; ++s) {
      mbar_init(smem_addr(&bars->q[s]), 128);
      for (int b = 0; b < 2; ++b) {
        mbar_init(smem_addr(&bars->s[s][b]), 1);
        mbar_init(smem_addr(&bars->p[s][b]), 128);
        mbar_init(smem_addr(&bars->o[s][b]), 1);
      }
    }
    mbar_init(smem_addr(&bars->idle), 1);
    bars->odd = 0;
    fence_mbar_init();
  }
  if (warp == kMmaWarp) tmem_alloc(smem_addr(&bars->tmem), kCols);
  Walk<MR> walk;
  const bool any = plan<MR, kThreads>(p, reinterpret_cast<PlanSmem<MR>*>(ring), &walk);
  grid_dep_launch_dependents();
  tmem_fence_before();
  __syncthreads();  // and the plan's scratch becomes the ring
  tmem_fence_after();
  if (!any) {
    if (warp == kMmaWarp) tmem_free(bars->tmem, kCols);
    return;
  }
  const uint32_t tmem = bars->tmem;
  const uint32_t ring_addr = smem_addr(ring), q_addr = smem_addr(qbuf);
  auto full = [&](int u) { return smem_addr(&bars->full[u]); };
  auto empty = [&](int u) { return smem_addr(&bars->empty[u]); };

  int before = 0;     // copying warps: units of the segments so far
  uint32_t done = 0;  // product warps: the stream's P tiles so far
  if (warp >= kLoadWarp && warp < kMmaWarp) {
    // ---------------------------------------------------------- copies
    uint32_t err = 0;
    Segment g;
    if constexpr (TMA) {
      // NS = 1: one warp copies K and V in the ring's order; NS = 2: one the Ks,
      // one the Vs (one for both took 1,000 cycles a unit, of which a pair of
      // tiles has two in some 1,300).  A lane holds the page id of one box, so a
      // load brings those of 32 / boxes tiles; the next chunk's is under way while
      // one is used, and Vs may still be in the one before.
      const int side = __shfl_sync(~0u, warp - kLoadWarp, 0);
      const int boxes = kTile / p.box;
      const uint32_t bytes = static_cast<uint32_t>(p.box) * L::kChunks * 128;
      while (true) {
        const bool more = walk.next(p, &g);
        const int n = __shfl_sync(~0u, more ? g.tile1 - g.tile0 : 0, 0);
        if (n == 0) break;
        const int tile0 = __shfl_sync(~0u, g.tile0, 0), end = __shfl_sync(~0u, g.kv_end, 0),
                  head = __shfl_sync(~0u, g.h, 0);
        const int32_t* table = a.table + g.r * a.table_stride;
        const int shift = __ffs(32 / boxes) - 1, per = 1 << shift;  // tiles of a chunk
        auto load_ids = [&](int chunk) {
          const int t = (tile0 + chunk * per) * kTile + lane * p.box;
          int id = 0;
          if (chunk * per < n && t < end) {
            id = __ldg(table + a.by_page.of(t));
            if (id < 0 || id >= a.num_blocks) err |= SV_DEVERR_PAGE, id = 0;
          }
          return id;
        };
        int chunk = 0, ids_before = 0, ids = load_ids(0), ids_after = load_ids(1);
        const int count = NS == 1 ? 2 * n : n;
        int ki = 0, vi = 0;
        for (int x = 0; x < count; ++x) {
          // the warp's next unit: whether it is a V, its tile and its place
          const bool val = NS == 2 ? side == 1 : ki == n || (ki >= 2 && ki == vi + 2);
          const int i = val ? vi++ : ki++;
          const int at = before + (val ? v_position(n, i) : k_position(i)), t0 = (tile0 + i) * kTile;
          if (i >> shift > chunk) {
            ++chunk;
            ids_before = ids, ids = ids_after, ids_after = load_ids(chunk + 1);
          }
          const int id = __shfl_sync(~0u, i >> shift == chunk ? ids : ids_before,
                                     (i & (per - 1)) * boxes + (lane / L::kChunks & (boxes - 1)));
          const int u = at % L::kUnits;
          if (at >= L::kUnits) mbar_wait(empty(u), (at / L::kUnits + 1) & 1, timed_out);
          __syncwarp();
          const int live = max(0, min(boxes, (end - t0 + p.box - 1) >> (__ffs(p.box) - 1)));
          if (elect_one()) mbar_arrive_expect_tx(full(u), live * bytes);
          const uint32_t dst = ring_addr + u * L::kUnitBytes;
          if (boxes == 1) {
            const int page = __shfl_sync(~0u, id, 0);  // for a uniform register
            const int in_page = t0 - a.by_page.of(t0) * a.page;
            if (live > 0 && elect_one()) {
#pragma unroll
              for (int c = 0; c < L::kChunks; ++c)
                tma_load4(dst + c * (kTile * 128), val ? &vmap : &kmap, c * 64, in_page, head, page,
                          full(u));
            }
          } else {  // several small pages: a lane a copy
            const int b = lane / L::kChunks, c = lane % L::kChunks;
            __syncwarp();
            if (b < live)
              tma_load4(dst + c * (kTile * 128) + b * p.box * 128, val ? &vmap : &kmap, c * 64, 0, head,
                        id, full(u));
          }
        }
        before += 2 * n;
      }
    } else if (warp == kLoadWarp) {
      // rows copied one by one, 16 bytes a lane: lane's addresses are those of rows
      // lane and lane + 32
      int issued = 0;
      constexpr int kPieces = DP / 8;
      while (walk.next(p, &g)) {
        const int32_t* table = a.table + g.r * a.table_stride;
        const int n = g.tile1 - g.tile0;
        int ki = 0, vi = 0;
        for (int x = 0; x < 2 * n; ++x, ++issued) {
          const bool val = ki == n || (ki >= 2 && ki == vi + 2);
          const int t0 = (g.tile0 + (val ? vi++ : ki++)) * kTile, u = issued % L::kUnits;
          const char* at[2];
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const int t = t0 + k * 32 + lane;
            at[k] = nullptr;
            if (t < g.kv_end) {
              const int page = a.by_page.of(t);
              int id = __ldg(table + page);
              if (id < 0 || id >= a.num_blocks) err |= SV_DEVERR_PAGE, id = 0;
              at[k] = (val ? a.v : a.k) + id * a.block + (t - page * a.page) * a.token +
                      g.h * a.head;
            }
          }
          if (issued >= L::kUnits) mbar_wait(empty(u), (issued / L::kUnits + 1) & 1, timed_out);
          __syncwarp();
          const uint32_t dst = ring_addr + u * L::kUnitBytes;
#pragma unroll
          for (int k = 0; k < 2; ++k)
            for (int i = 0; i < kPieces; ++i) {
              const int row = i * 32 / kPieces + lane / kPieces, j = lane % kPieces;
              const char* src = reinterpret_cast<const char*>(
                  __shfl_sync(~0u, reinterpret_cast<unsigned long long>(at[k]), row));
              const int rr = k * 32 + row;
              const bool on = src != nullptr && j * 8 < a.dim;
              cp_async16(dst + (j / 8) * (kTile * 128) + rr * 128 + (((j & 7) ^ (rr & 7)) << 4),
                         on ? src + j * 16 : a.k, on ? 16 : 0);
            }
          cp_async_commit();
          // the unit before the last has landed: hand it over
          if (issued >= 2) {
            cp_async_wait<2>();
            fence_async_smem();
            mbar_arrive(full((issued - 2) % L::kUnits));
          }
        }
      }
      if (issued >= 2) {
        cp_async_wait<1>();
        fence_async_smem();
        mbar_arrive(full((issued - 2) % L::kUnits));
      }
      cp_async_wait<0>();
      fence_async_smem();
      mbar_arrive(full((issued - 1) % L::kUnits));
    }
    if (err != 0 && a.dev_error != nullptr) atomicOr(a.dev_error, static_cast<int32_t>(err));
  } else if (warp >= kMmaWarp) {
    // ---------------------------------------------------------- products
    // One warp a stream: a wait takes some 150 cycles even where the phase is
    // over, and one warp for both streams spent more time in waits and issue than
    // the products take.  The whole warp walks, one lane issues.  What the
    // instructions' operands are formed from is the same in all lanes, and
    // shuffles say so to the compiler, which then keeps it in uniform registers:
    // operands moved there one by one took 80 cycles an instruction, against 48
    // (Q K^T, bound by reading Q and K from shared memory) and 64 (P V) of the
    // products themselves.
    constexpr uint32_t kQk = mma_idesc(kTile, false), kPv = mma_idesc(DP, true);
    const int s = __shfl_sync(~0u, warp - kMmaWarp, 0);
    const uint32_t tm = __shfl_sync(~0u, tmem, 0) + s * 2 * kTile,
                   to = __shfl_sync(~0u, tmem, 0) + kO + s * DP;
    int u = 0;
    uint32_t turn = 0;                     // parity of the ring's turn
    uint32_t tiles = 0;                    // the stream's S tiles so far
    uint32_t qturn = 0;
    auto step = [&]() {
      if (++u == L::kUnits) u = 0, turn ^= 1;
    };
    auto wait = [&](uint32_t bar, uint32_t parity) {
      mbar_wait(bar, parity, timed_out);
      __syncwarp();
      tmem_fence_after();
    };
    const uint64_t qdesc = smem_desc(q_addr, 0) + s * (L::kQBytes / 16),
                   kdesc = smem_desc(ring_addr, 0),
                   vdesc = smem_desc(ring_addr, DP > 64 ? kTile * 128 : 0);
    auto qk = [&]() {  // S from the K unit at u
      const uint32_t b = tiles & 1, d = tm + b * kTile;
      const uint64_t k = kdesc + u * (L::kUnitBytes / 16);
      if (elect_one()) {
#pragma unroll
        for (int i = 0; i < DP / 16; ++i)
          mma_ss(d, qdesc + (i / 4 * (kRows * 128) + i % 4 * 32) / 16,
                 k + (i / 4 * (kTile * 128) + i % 4 * 32) / 16, kQk, i > 0);
        mma_commit(empty(u));
        mma_commit(smem_addr(&bars->s[s][b]));
      }
      ++tiles;
      step();
    };
    Segment g;
    while (true) {
      const bool more = walk.next(p, &g);
      const int n = __shfl_sync(~0u, more ? g.tile1 - g.tile0 : 0, 0);
      if (n == 0) break;
      wait(smem_addr(&bars->q[s]), qturn);
      qturn ^= 1;
      if (s > 0 && __shfl_sync(~0u, g.rows <= kRows ? 1 : 0, 0)) {
        // no rows in this stream: its part in the ring, and its softmax may go on
        if (lane == 0) mbar_arrive(smem_addr(&bars->idle));
        for (int i = 0; i < 2 * n; ++i) {
          wait(full(u), turn);
          if (lane == 0) mbar_arrive(empty(u));
          step();
        }
        continue;
      }
      for (int i = 0; i < min(2, n); ++i) {
        wait(full(u), turn);
        qk();
      }
      for (int i = 0; i < n; ++i) {
        const uint32_t b = done & 1, pt = tm + b * kTile;
        const uint64_t v = vdesc + u * (L::kUnitBytes / 16);
        wait(full(u), turn);
        wait(smem_addr(&bars->p[s][b]), done >> 1 & 1);
        ++done;
        if (elect_one()) {
          mma_ts(to, pt, v, kPv, i > 0);
#pragma unroll
          for (int k = 1; k < kTile / 16; ++k) mma_ts(to, pt + k * 8, v + k * (2048 / 16), kPv, true);
          mma_commit(empty(u));
          mma_commit(smem_addr(&bars->o[s][b]));
        }
        step();
        if (i + 2 < n) {
          wait(full(u), turn);
          qk();
        }
      }
    }
  } else {
    // ---------------------------------------------------------- softmax
    const int st = warp >> 2;          // stream
    const int row = tid & 127;         // row of the stream's tile
    const int wrow = (warp & 3) * 32;  // the warp's first row
    const uint32_t lanes = static_cast<uint32_t>(wrow) << 16;
    const uint32_t s_at = tmem + lanes + st * 2 * kTile, o_at = tmem + lanes + kO + st * DP;
    // the stream's O up to tile t: S of tile t + 1 tells of tile t - 1, so at most
    // the last phase of this barrier can be open
    auto wait_o = [&](uint32_t t) {
      mbar_wait(smem_addr(&bars->o[st][t & 1]), t >> 1 & 1, timed_out);
      __syncwarp();
      tmem_fence_after();
    };
    const float c = fabsf(a.scale2);
    WarpWalk<MR>* const ww = walks + warp;
    uint32_t tiles = 0;  // the stream's tiles so far
    uint32_t idle = 0;   // parity of the next segment without rows here
    int u0 = 0;          // ring position of the segment's first unit, and its turn
    uint32_t turn0 = 0;
    // the walk's next segment, by lane 0, into shared memory (tile1 = -1: none)
    auto advance = [&]() {
      __syncwarp();
      if (lane == 0) {
        Walk<MR> w = ww->walk;
        Segment n;
        if (!w.next(p, &n)) n.tile1 = -1;
        ww->walk = w;
        ww->next = n;
      }
      __syncwarp();
    };
    // the next segment's query rows: lane's own row address, then 16-byte pieces
    auto load_q = [&]() {
      const Segment& n = ww->next;
      const int i = n.m * MR + st * kRows + wrow + lane;
      const char* src = nullptr;
      if (st * kRows + wrow + lane < n.rows)
        src = a.q + static_cast<int64_t>(n.row0 + a.by_group.of(i)) * a.q_row +
              static_cast<int64_t>(n.h * a.group + i - a.by_group.of(i) * a.group) * a.q_head;
      constexpr int kPieces = DP / 8;
      if (st * kRows + wrow < n.rows) {
#pragma unroll 4
        for (int k = 0; k < kPieces; ++k) {
          const int rr = k * 32 / kPieces + lane / kPieces, j = lane % kPieces;
          const char* from = reinterpret_cast<const char*>(
              __shfl_sync(~0u, reinterpret_cast<unsigned long long>(src), rr));
          const bool ok = from != nullptr && j * 8 < a.dim;
          cp_async16(q_addr + st * L::kQBytes + (j / 8) * (kRows * 128) + (wrow + rr) * 128 +
                         (((j & 7) ^ (rr & 7)) << 4),
                     ok ? from + j * 16 : a.q, ok ? 16 : 0);
        }
      }
      cp_async_commit();
    };

    if (lane == 0) ww->walk = walk;
    advance();
    load_q();
    while (ww->next.tile1 >= 0) {
      const Segment g = ww->next;
      cp_async_wait<0>();
      fence_async_smem();
      mbar_arrive(smem_addr(&bars->q[st]));
      const bool live = st * kRows < g.rows;         // the stream has rows
      const bool work = st * kRows + wrow < g.rows;  // the warp has rows
      const int pos = g.seq - g.l + a.by_group.of(g.m * MR + st * kRows + row);  // of this row
      const int lo = a.window > 0 ? max(0, pos - a.window + 1) : 0;
      // keys that every row of the item sees: [all_lo, all_hi)
      const int all_hi = g.seq - g.l + a.by_group.of(g.m * MR) + 1;
      const int all_lo = a.window > 0
          ? max(0, g.seq - g.l + a.by_group.of(g.m * MR + g.rows - 1) - a.window + 1) : 0;
      float m = -kInf, l = 0.0f;

      if (!live) {
        mbar_wait(smem_addr(&bars->idle), idle, timed_out);
        __syncwarp();
        idle ^= 1;
        advance();
        if (ww->next.tile1 >= 0) load_q();
      }
      for (int tile = g.tile0; live && tile < g.tile1; ++tile, ++tiles) {
        const int t0 = tile * kTile;
        const uint32_t buf = tiles & 1;
        const bool edge = t0 + kTile > all_hi || t0 < all_lo;
        mbar_wait(smem_addr(&bars->s[st][buf]), tiles >> 1 & 1, timed_out);
        __syncwarp();
        tmem_fence_after();
        if (tile + 1 == g.tile1) {  // the last S is formed: the query buffer is free
          advance();
          if (ww->next.tile1 >= 0) load_q();
        }
        if (edge) {  // set aside non-finite values that not all rows see; S is there,
                     // so the V unit's last occupant is gone and its turn is this one
          const int at_v = u0 + v_position(g.tile1 - g.tile0, tile - g.tile0);
          mbar_wait(full(at_v % L::kUnits), (turn0 ^ (at_v / L::kUnits)) & 1, timed_out);
          char* unit = ring + at_v % L::kUnits * L::kUnitBytes;
          uint32_t big = 0;  // the largest magnitude, NaN above all
#pragma unroll
          for (int at = row; at < L::kUnitBytes / 16; at += 128) {
            const uint4 v = *reinterpret_cast<const uint4*>(unit + at * 16);
            big = bf16x2_max_nan(big, bf16x2_max_nan(bf16x2_max_nan(v.x & 0x7fff7fffu, v.y & 0x7fff7fffu),
                                                     bf16x2_max_nan(v.z & 0x7fff7fffu, v.w & 0x7fff7fffu)));
          }
          if ((big & 0x7f80u) == 0x7f80u || (big & 0x7f800000u) == 0x7f800000u) {
            for (int at = row; at < L::kUnitBytes / 16; at += 128) {
              const int t = t0 + (at >> 3) % kTile;
              if (t >= all_lo && t < all_hi) continue;
              uint4 v = *reinterpret_cast<const uint4*>(unit + at * 16);
              uint32_t* w = reinterpret_cast<uint32_t*>(&v);
              bool odd = false;
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                if ((w[e] & 0x7f80u) == 0x7f80u) w[e] &= 0xffff0000u, odd = true;
                if ((w[e] & 0x7f800000u) == 0x7f800000u) w[e] &= 0xffffu, odd = true;
              }
              if (odd) {
                if (t < g.kv_end) bars->odd = 1;  // past it lies what no copy brought
                __threadfence_block();
                *reinterpret_cast<uint4*>(unit + at * 16) = v;
              }
            }
          }
          fence_async_smem();
        }
        if (work) {
          uint32_t x[kTile];
          tmem_ld32(s_at + buf * kTile, x);
          tmem_ld32(s_at + buf * kTile + 32, x + 32);
          tmem_wait_ld();
          float* s = reinterpret_cast<float*>(x);
          if (a.scale2 < 0.0f) {
#pragma unroll
            for (int k = 0; k < kTile; ++k) s[k] = -s[k];
          }
          if (edge) {
            const int from = lo - t0, to = pos + 1 - t0;
#pragma unroll
            for (int k = 0; k < kTile; ++k) s[k] = k >= from && k < to ? s[k] : -kInf;
          }
          float mx[4] = {m, s[0], s[1], s[2]};
          mx[3] = fmaxf(mx[3], s[3]);
#pragma unroll
          for (int k = 4; k < kTile; k += 8)
#pragma unroll
            for (int e = 0; e < 4 && k + 2 * e < kTile; ++e)
              mx[e] = fmaxf(fmaxf(mx[e], s[k + 2 * e]), s[k + 2 * e + 1]);
          const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
          if (tile == g.tile0) {
            m = top;
          } else {
            const bool rise = top > -kInf && (m == -kInf || (top - m) * c > kRescale);
            if (__any_sync(~0u, rise)) {
              const float f = top > m ? ex2((m - top) * c) : 1.0f;
              wait_o(tiles - 1);
#pragma unroll
              for (int k = 0; k < DP; k += 16) {
                uint32_t o[16];
                tmem_ld16(o_at + k, o);
                tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                tmem_st16(o_at + k, o);
              }
              l *= f;
              m = top;
            }
          }
          float base = m == -kInf ? 0.0f : m * c, mul = c;
          if (__any_sync(~0u, fabsf(base) > 0x1p20f)) {
            // scores so large that the rounding of m c would not cancel in s c - m c
#pragma unroll
            for (int k = 0; k < kTile; ++k) s[k] = (s[k] - (m == -kInf ? 0.0f : m)) * c;
            base = 0.0f, mul = 1.0f;
          }
          const uint64_t mul2 = pack2(mul, mul), base2 = pack2(-base, -base);
          uint64_t sum[2] = {0, 0};
#pragma unroll
          for (int k = 0; k < kTile; k += 32) {
            uint32_t w[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              float p0, p1;
              unpack2(fma2(pack2(s[k + 2 * e], s[k + 2 * e + 1]), mul2, base2), &p0, &p1);
              p0 = ex2(p0), p1 = ex2(p1);
              sum[e & 1] = add2(sum[e & 1], pack2(p0, p1));
              asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[e]) : "f"(p1), "f"(p0));
            }
            tmem_st16(s_at + buf * kTile + k / 2, w);
          }
          float s0, s1;
          unpack2(add2(sum[0], sum[1]), &s0, &s1);
          l += s0 + s1;
          tmem_wait_st();
        }
        tmem_fence_before();
        mbar_arrive(smem_addr(&bars->p[st][buf]));
      }
      u0 += 2 * (g.tile1 - g.tile0);
      turn0 ^= (u0 / L::kUnits) & 1;
      u0 %= L::kUnits;

      if (live) {
        // ------------------------------------------------------ epilogue
        wait_o(tiles - 1);
        if (work) {
          const bool valid = st * kRows + row < g.rows;
          const bool odd = *reinterpret_cast<volatile int32_t*>(&bars->odd) != 0;
          const int i = g.m * MR + st * kRows + row;
          const int head = g.h * a.group + i - a.by_group.of(i) * a.group;
          const int64_t orow = g.row0 + a.by_group.of(i);
          const int slot = 2 * blockIdx.x + (g.begins ? 1 : 0);
          const float inv = g.whole ? (l > 0.0f || l != l ? 1.0f / l : 0.0f) : 1.0f;
          const int prow = st * kRows + row;
#pragma unroll
          for (int k0 = 0; k0 < DP; k0 += 64) {
            uint32_t x[64];
            tmem_ld32(o_at + k0, x);
            tmem_ld32(o_at + k0 + 32, x + 32);
            tmem_wait_ld();
            float* o = reinterpret_cast<float*>(x);
            __syncwarp();
            if (!valid) continue;
            if (odd) {  // values set aside that this row sees
              for (int t = max(g.tile0 * kTile, lo); t < min(g.tile1 * kTile, pos + 1); ++t) {
                if (t >= all_lo && t < all_hi) {
                  t = min(all_hi, pos + 1) - 1;
                  continue;
                }
                const int page = a.by_page.of(t);
                int id = a.table[g.r * a.table_stride + page];
                if (id < 0 || id >= a.num_blocks) id = 0;
                const __nv_bfloat16* v = reinterpret_cast<const __nv_bfloat16*>(
                    a.v + id * a.block + (t - page * a.page) * a.token + g.h * a.head) + k0;
#pragma unroll
                for (int e = 0; e < 64; ++e)
                  if (k0 + e < a.dim && !(fabsf(__bfloat162float(v[e])) < kInf))
                    o[e] += __bfloat162float(v[e]);
              }
            }
            if (g.whole) {
              char* out = a.out + orow * a.o_row + head * a.o_head + k0 * 2;
#pragma unroll
              for (int e = 0; e < 64; e += 8) {
                uint4 w;
                asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w.x) : "f"(o[e + 1] * inv), "f"(o[e] * inv));
                asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w.y) : "f"(o[e + 3] * inv), "f"(o[e + 2] * inv));
                asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w.z) : "f"(o[e + 5] * inv), "f"(o[e + 4] * inv));
                asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w.w) : "f"(o[e + 7] * inv), "f"(o[e + 6] * inv));
                if (k0 + e < a.dim) *reinterpret_cast<uint4*>(out + e * 2) = w;
              }
            } else {
#pragma unroll
              for (int e = 0; e < 64; e += 4)
                p.o[(static_cast<int64_t>(slot) * (DP / 4) + (k0 + e) / 4) * MR + prow] =
                    make_float4(o[e], o[e + 1], o[e + 2], o[e + 3]);
            }
          }
          if (valid) {
            const float mc = m == -kInf ? -kInf : m * c;
            if (!g.whole)
              p.ml[static_cast<int64_t>(slot) * MR + prow] = make_float2(mc, l);
            else if (a.lse != nullptr)
              a.lse[orow * a.heads + head] = l > 0.0f || l != l ? (mc + log2f(l)) * kLn2 : -kInf;
          }
          tmem_fence_before();
        }
      }
    }
  }
  if (timed_out && a.dev_error != nullptr) atomicOr(a.dev_error, SV_DEVERR_TIMEOUT);
  tmem_fence_before();
  if (__syncthreads_or(timed_out)) {
    // Some warp gave up, and what it waited for may still be on its way: no copy
    // and no product outlives the CTA.  All are issued by now, so the last units
    // and the last product are each in the phase that is waited for.
    bool late = false;
    if (TMA && warp == kLoadWarp)
      for (int i = 0; i < L::kUnits && i < before; ++i) {
        const int at = before - 1 - i;
        mbar_wait(full(at % L::kUnits), (at / L::kUnits) & 1, late);
      }
    if (warp >= kMmaWarp && done > 0)
      mbar_wait(smem_addr(&bars->o[warp - kMmaWarp][(done - 1) & 1]), (done - 1) >> 1 & 1, late);
    __syncthreads();
  }
  tmem_fence_after();
  if (warp == kMmaWarp) tmem_free(tmem, kCols);
}

// ---------------------------------------------------------------- combine
//
// Joins the partials of the items that were cut.  Every block finds all of them
// from the workers' records and takes four rows at a time: the parts' weights
// 2^(m c - max) go to shared memory, then GROUPS threads sum four columns of a row,
// each over every GROUPS-th part, in worker order.  Bound by the latency of two rounds of loads,
// and by the partials' bytes (from L2) where there are many.
constexpr int kCombineRows = 4;

// threads of a group: four rows of DP / 4 columns, a whole number of warps per row
__host__ __device__ constexpr int combine_group(int dp) { return dp < 128 ? 128 : dp; }

template <int MR, int DP, int GROUPS, bool F32>
__global__ __launch_bounds__(GROUPS * combine_group(DP)) void attn_combine_kernel(const MmaArgs p,
                                                                                  int workers) {
  constexpr int kGroup = combine_group(DP), kCombineThreads = GROUPS * kGroup, kCombineGroups = GROUPS;
  __shared__ AttnRecord item[kMaxWorkers];
  __shared__ int32_t second[kMaxWorkers];  // the item's second worker
  __shared__ float4 sums[GROUPS > 1 ? GROUPS - 1 : 1][kGroup];
  __shared__ float weight[kCombineRows][kMaxWorkers], inverse[kCombineRows];
  __shared__ int32_t found[(kMaxWorkers + kCombineThreads - 1) / kCombineThreads * (kCombineThreads / 32)];
  const AttnArgs& a = p.a;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  grid_dep_wait();
  // the list is in worker order, the same in every block
  constexpr int kChunks = (kMaxWorkers + kCombineThreads - 1) / kCombineThreads;
  constexpr int kWarps = kCombineThreads / 32;
  AttnRecord mine[kChunks];
  unsigned vote[kChunks];
#pragma unroll
  for (int c = 0; c < kChunks; ++c) {
    const int w = c * kCombineThreads + tid;
    mine[c] = w < workers ? p.record[w] : AttnRecord{0, 0, 0, 0, 0};
  }
#pragma unroll
  for (int c = 0; c < kChunks; ++c) {
    vote[c] = __ballot_sync(~0u, mine[c].parts > 0);
    if (lane == 0) found[c * kWarps + warp] = __popc(vote[c]);
  }
  __syncthreads();
  int count = 0;
#pragma unroll
  for (int c = 0; c < kChunks; ++c)
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if (w == warp && mine[c].parts > 0) {
        const int at = count + __popc(vote[c] & ((1u << lane) - 1));
        item[at] = mine[c], second[at] = c * kCombineThreads + tid;
      }
      count += found[c * kWarps + w];
    }
  __syncthreads();
  for (int task = blockIdx.x; task < count * (MR / kCombineRows); task += gridDim.x) {
    const AttnRecord r = item[task % count];
    const int w0 = second[task % count] - 1, row0 = task / count * kCombineRows;
    const int rows = r.rows;
    if (row0 >= rows) continue;
    auto slot = [&](int i) { return static_cast<int64_t>(2 * (w0 + i) + (i == 0 ? 1 : 0)); };
    // thread: row row0 + tid % 4, columns [4 q, 4 q + 4), parts group, group + 4, ..;
    // the first parts' loads go out before the weights are known
    const int sub = tid % kCombineRows, q = tid / kCombineRows % (kGroup / 4), group = tid / kGroup,
              mine_row = row0 + sub;
    const bool on = mine_row < rows && q * 4 < a.dim;
    auto load = [&](int i) { return p.o[(slot(i) * (DP / 4) + q) * MR + mine_row]; };
    float4 x[8];
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (on && group + j * kCombineGroups < r.parts) x[j] = load(group + j * kCombineGroups);
    __syncthreads();  // the weights of the task before are done with
    if (warp < kCombineRows && row0 + warp < rows) {  // warp j: the weights of row row0 + j
      const int row = row0 + warp;
      float top = -kInf, l = 0.0f;
      for (int i = lane; i < r.parts; i += 32) top = fmaxf(top, p.ml[slot(i) * MR + row].x);
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, d));
      if (top == -kInf) top = 0.0f;
      for (int i = lane; i < r.parts; i += 32) {
        const float2 x = p.ml[slot(i) * MR + row];
        const float f = ex2(x.x - top);
        weight[warp][i] = f;
        l += x.y * f;
      }
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) l += __shfl_xor_sync(~0u, l, d);
      if (lane == 0) {
        inverse[warp] = l > 0.0f || l != l ? 1.0f / l : 0.0f;
        const int j = r.m * MR + row;
        if (a.lse != nullptr)
          a.lse[(static_cast<int64_t>(r.row0) + a.by_group.of(j)) * a.heads + r.h * a.group + j -
                a.by_group.of(j) * a.group] =
              l > 0.0f || l != l ? (top + log2f(l)) * kLn2 : -kInf;
      }
    }
    __syncthreads();
    float4 o = make_float4(0, 0, 0, 0);
    for (int i = group; i < r.parts; i += 8 * kCombineGroups) {
      if (i > group) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (on && i + j * kCombineGroups < r.parts) x[j] = load(i + j * kCombineGroups);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (on && i + j * kCombineGroups < r.parts) {
          const float f = weight[sub][i + j * kCombineGroups];
          o.x = fmaf(x[j].x, f, o.x), o.y = fmaf(x[j].y, f, o.y);
          o.z = fmaf(x[j].z, f, o.z), o.w = fmaf(x[j].w, f, o.w);
        }
    }
    if (GROUPS > 1) {
      if (group > 0) sums[group - 1][tid % kGroup] = o;
      __syncthreads();
    }
    if (on && group == 0) {
#pragma unroll
      for (int j = 0; j < kCombineGroups - 1; ++j) {
        const float4 y = sums[j][tid];
        o.x += y.x, o.y += y.y, o.z += y.z, o.w += y.w;
      }
      const float inv = inverse[sub];
      const int j = r.m * MR + mine_row;
      const int64_t orow = static_cast<int64_t>(r.row0) + a.by_group.of(j);
      const int head = r.h * a.group + j - a.by_group.of(j) * a.group;
      char* out = a.out + orow * a.o_row + head * a.o_head;
      if constexpr (F32) {
        *reinterpret_cast<float4*>(out + q * 16) =
            make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv);
      } else {
        uint2 v;
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(v.x) : "f"(o.y * inv), "f"(o.x * inv));
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(v.y) : "f"(o.w * inv), "f"(o.z * inv));
        *reinterpret_cast<uint2*>(out + q * 8) = v;
      }
    }
  }
}

}  // namespace serve
}  // namespace sv
