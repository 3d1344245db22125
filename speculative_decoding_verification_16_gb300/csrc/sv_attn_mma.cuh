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
// Caches of 8 bits: codes come by the same copies, and warps of their own turn them into
// fp16 operands in place (turn_codes, below), so queries and weights are fp16 there too.
// Decoding is bound by those warps and by shared memory, not by the half as many bytes:
// 64 single tokens, 64/8 heads of 128, 2,048 to 32,768 cached, 397 us (3.9 TB/s, 0.57 of
// the copy rate); 32 x 16 tokens 153 us; 3 chunks of 2,048 760 us (1.02 PFLOP/s), where
// the softmax and the codes share the issue slots.  The kernel's hot loops barely fit the
// instruction cache: unrolling one of them moved the chunks by up to a third.
//
// Trees: TREE replaces the causal limit by a row's mask in the tiles that hold the
// request's own tokens; the context's tiles are as ever.  32 trees of up to 64 tokens over
// 512 to 16,384, 32/8 heads, 126 us; one of 64 over 4,000 27 us.
//
// Masked places.  S of a masked key is replaced, whatever it holds.  A masked
// value is multiplied by P = 0, so a NaN or infinity there would reach every
// row: in the tiles that not all rows see whole, V's non-finite elements under
// keys that some row does not see are set to 0 in shared memory, and the
// epilogue adds them, from the cache, to the rows that do see them.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>

#include "sv_attn_args.cuh"
#include "sv_e4m3.cuh"
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
  int32_t over;           // what an item costs beside its tiles, in tiles (below)
  AttnRecord* record;     // [kMaxWorkers]
  float2* ml;             // [2 * kMaxWorkers][rows]: m c (of codes r) and l of the partials
  float4* o;              // [2 * kMaxWorkers][DP / 4][rows]
};

constexpr int kMaxUnits = 10;
__host__ __device__ constexpr int attn_units(int ns, int dp) { return ns == 1 && dp >= 128 ? 5 : kMaxUnits; }
// CTAs an SM.
__host__ __device__ constexpr int attn_per_sm(int ns, int dp) { return ns == 1 && dp <= 128 ? 2 : 1; }
// Where keys and values come from: copies of single rows or tensor copies of page
// pieces, of bf16 or of codes of 8 bits, which warps turn into fp16 in place.
constexpr int kRowCopies = 0, kTensorCopies = 1, kCodeRows = 2, kCodeTensor = 3;
__host__ __device__ constexpr bool of_codes(int src) { return src >= kCodeRows; }
// Warps that turn codes into operands.  One stream: eight warps a CTA, two CTAs an SM, 128
// registers a thread, which the softmax needs; a ninth warp would leave one CTA an SM, since
// registers are a quarter SM's (64 single tokens 581 us).  Two streams: 16 warps.
__host__ __device__ constexpr int attn_turners(int ns, int dp, int src) {
  return !of_codes(src) ? 0 : ns == 2 ? 4 : 2;
}
// softmax, products, copies, codes
__host__ __device__ constexpr int attn_threads(int ns, int dp, int src) {
  return (ns * 6 + attn_turners(ns, dp, src)) * 32;
}
constexpr int kBarBytes = 448;
// query tiles, ring of key and value tiles, barriers, the softmax warps' walks
__host__ __device__ constexpr int attn_smem(int ns, int dp) {
  return ns * kRows * dp * 2 + attn_units(ns, dp) * kTile * dp * 2 + kBarBytes + ns * 4 * 104;
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
  int n;  // its share of the work: the tiles and what it costs beside, or 1 where items
          // are not cut
};

// EXT, here and below: a call over codes or of trees, whose items cost `over` beside their
// tiles and may have masks.  Other calls do without either: formed in their plan and walks
// too, they took one block over 4,000 keys from 15.8 to 16.4 us, 32 x 16 tokens from 162 to
// 165, chunks of 4,096 from 1,255 to 1,272.
template <int MR, bool EXT>
__device__ __forceinline__ ItemTiles item_tiles(const MmaArgs& p, const Span& s, int m) {
  const AttnArgs& a = p.a;
  ItemTiles t;
  const int all = s.l * a.group;
  t.rows = min(MR, all - m * MR);
  const int j0 = a.by_group.of(m * MR), j1 = a.by_group.of(m * MR + t.rows - 1);
  t.kv_end = max(0, s.seq - s.l + j1 + 1);
  // a tree's rows may all lie at its root's position
  const int kv_lo = a.window > 0 ? max(0, s.seq - s.l + (EXT && a.mask != nullptr ? 0 : j0) - a.window + 1) : 0;
  t.lo = kv_lo / kTile;
  t.tiles = max(1, (t.kv_end + kTile - 1) / kTile - t.lo);
  t.n = p.whole ? 1 : t.tiles + (EXT ? p.over : 0);
  return t;
}

template <int MR, bool EXT>
__device__ __forceinline__ int64_t head_tiles(const MmaArgs& p, const Span& s) {
  int64_t n = 0;
  if (s.l > 0)
    for (int m = 0; m * MR < s.l * p.a.group; ++m) n += item_tiles<MR, EXT>(p, s, m).n;
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

// An item counts `over` units before its tiles: query rows, a pipeline filled and drained,
// results written cost a worker as much, and workers with many short items ended late
// (32 requests of 16 tokens over 512 to 32,768 in 8 bits: the last after 209 us, the mean
// 145).  A run that ends within these units leaves the item to the next worker, which
// starts it from its first tile.
template <int MR, bool EXT>
struct Walk {  // a worker's segments in order
  int r, h, m, off;
  int64_t left;
  Span s;

  // What is left ends before the next item's tiles.
  __device__ __forceinline__ bool idle(const MmaArgs& p) const {
    return EXT && off == 0 && !p.whole && left <= p.over;
  }
  __device__ __forceinline__ bool next(const MmaArgs& p, Segment* g) {
    if (left <= 0) return false;
    if (idle(p)) {
      left = 0;
      return false;
    }
    const ItemTiles t = item_tiles<MR, EXT>(p, s, m);
    const int over = EXT ? p.over : 0;
    const int take = static_cast<int>(min(left, static_cast<int64_t>(t.n - off)));
    g->r = r, g->h = h, g->m = m, g->row0 = s.row0, g->l = s.l, g->seq = s.seq;
    g->tile0 = t.lo + (EXT ? max(0, off - over) : off), g->tile1 = t.lo + (p.whole ? t.tiles : off + take - over);
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
          if (left > 0) do s = span_of<EXT>(p.a, ++r); while (s.l <= 0);
        }
      }
    }
    return true;
  }
};

template <int MR, bool EXT>
struct PlanSmem {
  int64_t part[16];
  Walk<MR, EXT> walk;
};

// Every CTA finds its own run from the requests' lengths: a scan over the
// requests' tiles, then the thread whose request holds the run's start sets out
// the walk.  More requests than threads: the tiles are formed twice, once for the
// total and once up to the start.
template <int MR, int THREADS, bool EXT>
__device__ __forceinline__ bool plan(const MmaArgs& p, PlanSmem<MR, EXT>* sm, Walk<MR, EXT>* w) {
  const AttnArgs& a = p.a;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  constexpr int kW = THREADS / 32;
  Span s{0, 0, 0};
  int64_t mine = 0, per_head = 0;
  bool bad = false;
  for (int r = tid; r < a.B; r += THREADS) {
    s = span_of<EXT>(a, r, &bad);
    per_head = head_tiles<MR, EXT>(p, s);
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
    Walk<MR, EXT> x;
    x.r = r, x.s = s;
    x.h = rem < (1 << 30) && per_head < (1 << 30)
              ? static_cast<int>(static_cast<uint32_t>(rem) / static_cast<uint32_t>(per_head))
              : static_cast<int>(rem / per_head);
    rem -= x.h * per_head;
    x.m = 0;
    ItemTiles t = item_tiles<MR, EXT>(p, s, 0);
    while (rem >= t.n) rem -= t.n, t = item_tiles<MR, EXT>(p, s, ++x.m);
    x.off = static_cast<int>(rem);
    x.left = worker_start(total, workers, me + 1) - start;
    if (EXT && !p.whole && x.off <= p.over) x.left += x.off, x.off = 0;  // from the first tile
    sm->walk = x;
    item = t.n;
  };
  if (a.B <= THREADS) {
    if (before <= start && start < before + mine) set_out(tid, start - before);
  } else {
    int64_t carry = 0;
    for (int base = 0; base < a.B && carry <= start; base += THREADS) {
      const int r = base + tid;
      s = r < a.B ? span_of<EXT>(a, r) : Span{0, 0, 0};
      per_head = head_tiles<MR, EXT>(p, s);
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
    int begins = worker_of(total, workers, first);  // the item's first worker
    while (EXT && w->off > 0 && worker_start(total, workers, begins + 1) - first <= p.over) ++begins;
    if (w->off > 0 && begins == me - 1)
      rec = AttnRecord{worker_of(total, workers, first + item - 1) - me + 2,
                       item_tiles<MR, EXT>(p, w->s, w->m).rows, w->s.row0, w->h, w->m};
    p.record[me] = rec;
  }
  return !w->idle(p);
}

// ---------------------------------------------------------------- trees
//
// Row j of a tree sees the context's keys, less those that its window leaves behind
// (its own position is ctx + its depth), and of the request's rows up to itself those
// that its mask names.  `p` is ctx + j, the place of the row's key in the cache.
__device__ __forceinline__ int tree_lo(const AttnArgs& a, const Segment& g, int p) {
  const int ctx = g.seq - g.l;
  if (a.window <= 0 || p - ctx >= g.l) return 0;
  const int pos = max(ctx, min(__ldg(a.positions + g.row0 + (p - ctx)), g.seq - 1));
  return min(ctx, max(0, pos - a.window + 1));
}
// Keys from here up to the context's end are seen by every row.
__device__ __forceinline__ int tree_all_lo(const AttnArgs& a, const Segment& g) {
  return a.window > 0 ? min(g.seq - g.l, max(0, g.seq - a.window)) : 0;
}
// Whether the row sees key t <= p that its window leaves it.
__device__ __forceinline__ bool tree_sees(const AttnArgs& a, const Segment& g, int p, int t) {
  const int ctx = g.seq - g.l, i = t - ctx;
  return i < 0 || (__ldg(a.mask + static_cast<int64_t>(g.row0 + (p - ctx)) * a.mask_words + (i >> 5)) >> (i & 31) & 1) != 0;
}
// The same of the 64 keys from t0, with the window and the row's own place: bit k.
__device__ __forceinline__ uint64_t tree_bits(const AttnArgs& a, const Segment& g, int p, int lo, int t0) {
  const int ctx = g.seq - g.l, first = t0 - ctx;
  uint64_t bits = ~uint64_t{0};
  if (first > -64) {
    const uint32_t* row = a.mask + static_cast<int64_t>(g.row0 + (p - ctx)) * a.mask_words;
    auto word = [&](int w) { return w < a.mask_words ? __ldg(row + w) : 0u; };
    const int w = max(first, 0) >> 5, shift = max(first, 0) & 31;
    const uint32_t x = word(w), y = word(w + 1), z = word(w + 2);
    bits = static_cast<uint64_t>(__funnelshift_r(y, z, shift)) << 32 | __funnelshift_r(x, y, shift);
    if (first < 0) bits = bits << -first | ((uint64_t{1} << -first) - 1);
  }
  const int n = p + 1 - t0;  // keys up to the row's own
  if (n < 64) bits &= n > 0 ? (uint64_t{1} << n) - 1 : 0;
  if (lo > t0) bits &= lo - t0 < 64 ? ~uint64_t{0} << (lo - t0) : 0;
  return bits;
}

// ---------------------------------------------------------------- codes
//
// Codes become fp16 operands, two instructions a pair (bf16 took six: there is no direct
// conversion).  fp16 holds every code exactly, but not every power of two, so a tile's
// powers are taken relative to 2^E, 2^7 below its largest: the rows' factors
// 2^(exp - E) are at most 2^7, exact down to 2^-15, 2^-22 of the largest; below, half of
// fp16's smallest step may be lost, 2^-25 2^E, and rows of factors below 2^-24 are taken
// for zeros.  Queries are brought into fp16's range by a power of two a row, 2^qe: its
// largest element to [2^14, 2^15), so elements down to 2^-31 of the largest are exact and
// smaller ones lose at most 2^-25, 2^-39 of it.  The keys' E and qe scale the tile's scores.
//
// Values of far apart E need references of their own for O and l: the key that counts
// most in O, by s c + E, may count nothing in l, which knows no E, and the other way.  Of
// a row r is the largest product q k so far (raised late, by 2^60), l is the sum of
// 2^((q k - r) c), and O is held for the reference r c + D, D from the largest
// s c + E - 7 = r c + D: a tile's weights are w = 2^(s c + E - r c - D), near 2^7 where they
// count, O += w (v 2^-E) and l += 2^(D - E) w.  Where a tile's weights all lie below 2^-53,
// their part of l is formed without E and D.  Weights in fp16 have 11 bits, bf16's 8; the
// row's largest is at least 2^7 (kLift; and at most 2^15, O being rescaled late), and what
// fp16 loses of a small one is at most 2^-25, 2^-32 of the largest.  A partial is O
// 2^D / l, the part's own mean, with r and l.  (One reference for both, and l with 2^-E in
// it: where E rose by 126 from one tile to the next, l lost the tiles before.)
constexpr float kLift = 7.0f;
constexpr int kFactorMin = -87;  // least E: 2^D / l stays a normal number
constexpr float kRaise = 60.0f;  // log2 of how far l's terms may exceed 1
constexpr float kApart = 60.0f;
constexpr float kLargeScore = 1024.0f;  // of |r c|, above which r c + D - E is off by more than 2^-14
// E of a tile whose rows' largest exponent is `most`.
__device__ __forceinline__ int tile_exponent(int most) { return max(most - 7, kFactorMin); }

__device__ __forceinline__ uint32_t code_pair(uint32_t c, uint32_t f) {  // the low half's two codes
  uint32_t h, d;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(c)));
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(h), "r"(f));
  return d;
}
__device__ __forceinline__ uint32_t code_factor(int d) {  // 2^d twice, d <= 7
  const uint32_t h = d >= -14 ? static_cast<uint32_t>(max(d, -14) + 15) << 10 : d >= -24 ? 1u << (max(d, -24) + 24) : 0u;
  return h * 0x10001u;
}
__device__ __forceinline__ float pow2_any(int e) {  // 2^e, e in [-149, 127]
  return __uint_as_float(e >= -126 ? static_cast<uint32_t>(e + 127) << 23 : 0x400000u >> (-127 - e));
}
// x 2^e, e in [-252, 254]: two factors of one sign
__device__ __forceinline__ float scaled(float x, int e) { return x * pow2(e >> 1) * pow2(e - (e >> 1)); }

// ---------------------------------------------------------------- kernel
template <int NS, int DP>
struct AttnSmem {
  static constexpr int kUnits = attn_units(NS, DP);
  static constexpr int kUnitBytes = kTile * DP * 2;
  static constexpr int kQBytes = kRows * DP * 2;
  static constexpr int kChunks = DP / 64;
};

struct AttnBars {
  uint64_t full[kMaxUnits], empty[kMaxUnits], raw[kMaxUnits];  // raw: codes are there
  uint64_t q[2], s[2][2], p[2][2], o[2][2], idle;  // by stream; s, p and o by S buffer too
  int32_t key_exp[8];  // of codes: E of a tile's keys
  float value_exp[8];  // and values
  uint32_t tmem;
  int32_t odd;  // a non-finite value was set aside in this CTA
};
static_assert(sizeof(AttnBars) <= kBarBytes, "barrier block");

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

template <int MR, bool EXT>
struct WarpWalk {
  Walk<MR, EXT> walk;
  Segment next;
};

// One of the warps that turn codes into operands.  It takes every kTurners-th tile,
// keys and values.  Codes lie in the unit itself: those of 128 columns (64 of a narrow
// head) in the rows of the second of the two chunks that they become, so a row is read
// and then written over, and no other place is needed.  Each byte of a cache passes
// through shared memory six times (copied in, read, written twice over, read twice over
// by the product), which bounds decoding: with the query's re-reads 1,024 cycles a tile
// of 64 keys.  A quarter warp takes 64 columns of rows r and r ^ 5, for which the swizzle
// spreads both the reads of codes and the writes of operands over all banks (rows of 64
// codes are not swizzled: r and r + 1).  The exponents of a tile's rows are read a tile
// ahead, the page ids two.
struct CodeTile {
  bool some;
  uint32_t at[2];      // its units' numbers in the CTA's ring: keys, values
  int tile;            // its number in the CTA
  int head;
  int in_page[2];      // lane's rows lane and lane + 32: the place in the page
  int id[2];           // and the page
};

template <int NS, int DP, int TURNERS, typename Raw, typename Full, typename Empty>
__device__ __forceinline__ void turn_codes(const MmaArgs& p, Walk<NS * kRows, true> walk, int warp, int lane,
                                           char* ring, AttnBars* bars, Raw raw, Full full, Empty empty,
                                           bool& timed_out) {
  using L = AttnSmem<NS, DP>;
  // Waits tell phases by their parity, so the phase before must be over: of a copy it is
  // when the buffer's last unit is released, which is waited for first; of that release
  // it is because the warp's last unit lies less than a ring before this one and units
  // are released in order.
  static_assert(2 * TURNERS - 1 <= L::kUnits && L::kUnits >= 3, "a warp's next unit is within a turn of its last");
  const AttnArgs& a = p.a;
  Segment g;
  int n = 0;             // the segment's tiles
  int i = warp;          // the warp's next tile in it
  int before = 0;        // tiles of the segments before it
  auto plan_tile = [&](CodeTile* u) {  // the warp's next tile, its page ids under way
    while (i >= n) {
      before += n;
      i -= n;
      n = walk.next(p, &g) ? g.tile1 - g.tile0 : 0;
      if (n == 0) {
        u->some = false;
        return;
      }
    }
    u->some = true;
    u->at[0] = 2 * before + k_position(i), u->at[1] = 2 * before + v_position(n, i);
    u->tile = before + i;
    u->head = g.h;
    const int t0 = (g.tile0 + i) * kTile;
    const int32_t* table = a.table + g.r * a.table_stride;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      // rows behind the last key: its factor again, for what no row of the item sees
      const int t = max(0, min(t0 + k * 32 + lane, g.kv_end - 1)), page = a.by_page.of(t);
      u->in_page[k] = t - page * a.page;
      u->id[k] = 0;
      if (g.kv_end > 0) u->id[k] = __ldg(table + page);
    }
    i += TURNERS;
  };
  // the exponents of lane's rows, keys' and values', under way
  auto exponents = [&](const CodeTile& u, int* exp) {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int id = static_cast<uint32_t>(u.id[k]) < static_cast<uint32_t>(a.num_blocks) ? u.id[k] : 0;
      const int64_t at = static_cast<int64_t>(id) * a.e_block + static_cast<int64_t>(u.in_page[k]) * a.e_token +
                         static_cast<int64_t>(u.head) * a.e_head;
      exp[k] = __ldg(a.k_exps + at), exp[2 + k] = __ldg(a.v_exps + at);
    }
  };
  // lane's place in a load of 512 bytes
  constexpr int kPairs = DP == 64 ? 4 : 2, kSteps = kTile / (2 * kPairs), kStepsAtOnce = kSteps / 2;
  const int unit16 = lane & 3, second = lane >> 2 & 1, chunk = DP == 64 ? 0 : lane >> 3 & 1,
            pair = DP == 64 ? lane >> 3 : lane >> 4;

  CodeTile cur, next, after;
  cur.some = next.some = false, after.some = true;
  int exp[4] = {0, 0, 0, 0}, next_exp[4] = {0, 0, 0, 0};
  for (int stage = 0; stage < 2 || cur.some; ++stage) {  // the first two fill the pipeline
    if (next.some) exponents(next, next_exp);
    if (after.some) plan_tile(&after);
    if (stage >= 2) {
      const int ek = tile_exponent(__reduce_max_sync(~0u, max(exp[0], exp[1]))),
                ev = tile_exponent(__reduce_max_sync(~0u, max(exp[2], exp[3])));
#pragma unroll 1
      for (int val = 0; val < 2; ++val) {
        const int e0 = val != 0 ? exp[2] - ev : exp[0] - ek, e1 = val != 0 ? exp[3] - ev : exp[1] - ek;
        const uint32_t f[2] = {code_factor(e0), code_factor(e1)};
        const uint32_t at = val != 0 ? cur.at[1] : cur.at[0], u = at % L::kUnits, turn = at / L::kUnits;
        if (turn > 0) mbar_wait(empty(u), (turn + 1) & 1, timed_out);
        mbar_wait(raw(u), turn & 1, timed_out);
        __syncwarp();
        // read when the tile's scores are formed.  The slot's last tile is done with: its
        // values' unit lies before the one just released
        if (val == 0 && lane == 0)
          bars->key_exp[cur.tile & 7] = ek, bars->value_exp[cur.tile & 7] = static_cast<float>(ev);
        char* const unit = ring + u * L::kUnitBytes;
#pragma unroll
        for (int part = 0; part < (DP == 256 ? 2 : 1); ++part) {
          char* const out = unit + part * (2 * kTile * 128);
          const char* const in = out + (DP == 64 ? kTile * 64 : kTile * 128);
#pragma unroll 1
          for (int half = 0; half < 2; ++half) {
            const uint32_t fh = half == 0 ? f[0] : f[1];
#pragma unroll
            for (int i0 = 0; i0 < kSteps / 2; i0 += kStepsAtOnce) {
              uint4 c[kStepsAtOnce];
              int row[kStepsAtOnce];
#pragma unroll
              for (int e = 0; e < kStepsAtOnce; ++e) {
                const int step = i0 + e;  // of the half
                if constexpr (DP == 64) {
                  row[e] = half * 32 + step * 8 + pair * 2 + second;
                  c[e] = *reinterpret_cast<const uint4*>(in + row[e] * 64 + unit16 * 16);
                } else {
                  const int r = (step & 1) * 2 + pair;
                  row[e] = half * 32 + (step >> 1) * 8 + (second != 0 ? r ^ 5 : r);
                  c[e] = *reinterpret_cast<const uint4*>(in + row[e] * 128 + (((chunk * 4 + unit16) ^ (row[e] & 7)) << 4));
                }
              }
              __syncwarp();  // all have read before any writes
#pragma unroll
              for (int e = 0; e < kStepsAtOnce; ++e) {
                const uint32_t s = __shfl_sync(~0u, fh, row[e] & 31);
                char* const to = out + chunk * (kTile * 128) + row[e] * 128;
                *reinterpret_cast<uint4*>(to + (((unit16 * 2) ^ (row[e] & 7)) << 4)) =
                    make_uint4(code_pair(c[e].x, s), code_pair(c[e].x >> 16, s), code_pair(c[e].y, s), code_pair(c[e].y >> 16, s));
                *reinterpret_cast<uint4*>(to + (((unit16 * 2 + 1) ^ (row[e] & 7)) << 4)) =
                    make_uint4(code_pair(c[e].z, s), code_pair(c[e].z >> 16, s), code_pair(c[e].w, s), code_pair(c[e].w >> 16, s));
              }
            }
          }
        }
        fence_async_smem();
        mbar_arrive(full(u));
      }
    }
    cur = next, next = after;
#pragma unroll
    for (int k = 0; k < 4; ++k) exp[k] = next_exp[k];
  }
}

// The first `rows` rows of a warp's 32 of a query tile brought from bf16 into fp16's
// range in place, a row's largest element to [2^14, 2^15), and negated where the scale is
// negative.  Returns log2 of what lane's row was divided by.  DP / 8 lanes a row, few
// instructions: run once an item, they come from far away.
template <int DP>
__device__ __forceinline__ int query_to_fp16(char* tile, int lane, int rows, bool negated) {
  constexpr int kLanes = DP / 8, kEach = 32 / kLanes;  // of a row; rows at once
  constexpr int kFlight = 4;                           // such steps together
  const int j = lane % kLanes, sub = lane / kLanes;
  char* const at = tile + (j >> 3) * (kRows * 128);
  int mine = 0;
#pragma unroll 1
  for (int r0 = 0; r0 < rows; r0 += kFlight * kEach) {
    uint4 v[kFlight];
    int top[kFlight];
    auto unit = [&](int i) {
      const int row = r0 + i * kEach + sub;
      return reinterpret_cast<uint4*>(at + row * 128 + (((j & 7) ^ (row & 7)) << 4));
    };
#pragma unroll
    for (int i = 0; i < kFlight; ++i) v[i] = *unit(i);
#pragma unroll
    for (int i = 0; i < kFlight; ++i) {  // the largest biased exponent
      const uint32_t big = bf16x2_max_nan(bf16x2_max_nan(v[i].x & 0x7fff7fffu, v[i].y & 0x7fff7fffu),
                                          bf16x2_max_nan(v[i].z & 0x7fff7fffu, v[i].w & 0x7fff7fffu));
      top[i] = max(static_cast<int>(big >> 7 & 0xff), static_cast<int>(big >> 23));
    }
#pragma unroll
    for (int d = kLanes / 2; d > 0; d >>= 1)
#pragma unroll
      for (int i = 0; i < kFlight; ++i) top[i] = max(top[i], __shfl_xor_sync(~0u, top[i], d));
#pragma unroll
    for (int i = 0; i < kFlight; ++i) {
      const int e = max(14, min(top[i], 254));  // 255: not finite, whatever the factor
      const float f = negated ? -pow2_any(141 - e) : pow2_any(141 - e);
      uint32_t* w = reinterpret_cast<uint32_t*>(&v[i]);
#pragma unroll
      for (int k = 0; k < 4; ++k)
        asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(w[k]) : "f"(bf16hi(w[k]) * f), "f"(bf16lo(w[k]) * f));
      *unit(i) = v[i];
      const int other = __shfl_sync(~0u, e, lane % kEach * kLanes);  // of the step's row lane % kEach
      if (lane / kEach == r0 / kEach + i) mine = other - 141;
    }
  }
  return mine;
}

template <int NS, int DP, int SRC, bool TREE>
__global__ __launch_bounds__(attn_threads(NS, DP, SRC), attn_per_sm(NS, DP)) void attn_mma_kernel(
    const MmaArgs p, const __grid_constant__ CUtensorMap kmap,
    const __grid_constant__ CUtensorMap vmap) {
  using L = AttnSmem<NS, DP>;
  constexpr int MR = NS * kRows;
  constexpr int kThreads = attn_threads(NS, DP, SRC), kTurners = attn_turners(NS, DP, SRC);
  constexpr bool TMA = SRC == kTensorCopies || SRC == kCodeTensor, CODES = of_codes(SRC),
                 EXT = CODES || TREE;
  // a unit as it is copied: chunks of columns side by side, each of 64 rows
  constexpr int kCopyChunks = !CODES ? L::kChunks : DP == 256 ? 2 : 1;
  constexpr int kCopyRow = CODES && DP == 64 ? 64 : 128;  // bytes of a row of a chunk
  constexpr int kCopyCols = CODES ? kCopyRow : 64;
  constexpr int kCopyAt = !CODES ? 0 : kTile * kCopyRow;  // where the first lies in the unit
  constexpr int kCopyStep = (CODES ? 2 : 1) * kTile * 128;
  constexpr uint32_t kCols = attn_per_sm(NS, DP) == 2 ? 256 : 512;
  // tensor memory columns: two S buffers of each stream, then O of each
  constexpr uint32_t kO = NS * 2 * kTile;
  extern __shared__ __align__(1024) char smem[];
  const AttnArgs& a = p.a;
  char* const qbuf = smem;
  char* const ring = smem + NS * L::kQBytes;
  AttnBars* const bars = reinterpret_cast<AttnBars*>(ring + L::kUnits * L::kUnitBytes);
  WarpWalk<MR, EXT>* const walks = reinterpret_cast<WarpWalk<MR, EXT>*>(reinterpret_cast<char*>(bars) + kBarBytes);
  static_assert(sizeof(WarpWalk<MR, EXT>) <= 104, "walk block");
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  constexpr int kSoftmax = NS * 4, kLoadWarp = kSoftmax, kMmaWarp = kSoftmax + NS,
                kTurnWarp = kMmaWarp + NS;
  bool timed_out = false;

  if (tid == 0) {
    for (int i = 0; i < L::kUnits; ++i) {
      mbar_init(smem_addr(&bars->full[i]), CODES || !TMA ? 32 : 1);
      if constexpr (CODES) mbar_init(smem_addr(&bars->raw[i]), TMA ? 1 : 32);
      mbar_init(smem_addr(&bars->empty[i]), NS);
    }
    for (int s = 0; s < NS; ++s) {
      mbar_init(smem_addr(&bars->q[s]), 128);
      for (int b = 0; b < 2; ++b) {
        mbar_init(smem_addr(&bars->s[s][b]), CODES ? 2 : 1);
        mbar_init(smem_addr(&bars->p[s][b]), 128);
        mbar_init(smem_addr(&bars->o[s][b]), 1);
      }
    }
    mbar_init(smem_addr(&bars->idle), 1);
    bars->odd = 0;
    fence_mbar_init();
  }
  if (warp == kMmaWarp) tmem_alloc(smem_addr(&bars->tmem), kCols);
  Walk<MR, EXT> walk;
  const bool any = plan<MR, kThreads, EXT>(p, reinterpret_cast<PlanSmem<MR, EXT>*>(ring), &walk);
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
  auto copied = [&](int u) { return smem_addr(CODES ? &bars->raw[u] : &bars->full[u]); };

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
      const uint32_t bytes = static_cast<uint32_t>(p.box) * kCopyChunks * kCopyRow;
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
                                     (i & (per - 1)) * boxes + (lane / kCopyChunks & (boxes - 1)));
          const int u = at % L::kUnits;
          if (at >= L::kUnits) mbar_wait(empty(u), (at / L::kUnits + 1) & 1, timed_out);
          __syncwarp();
          const int live = max(0, min(boxes, (end - t0 + p.box - 1) >> (__ffs(p.box) - 1)));
          if (elect_one()) mbar_arrive_expect_tx(copied(u), live * bytes);
          const uint32_t dst = ring_addr + u * L::kUnitBytes + kCopyAt;
          if (boxes == 1) {
            const int page = __shfl_sync(~0u, id, 0);  // for a uniform register
            const int in_page = t0 - a.by_page.of(t0) * a.page;
            if (live > 0 && elect_one()) {
#pragma unroll
              for (int c = 0; c < kCopyChunks; ++c)
                tma_load4(dst + c * kCopyStep, val ? &vmap : &kmap, c * kCopyCols, in_page, head, page,
                          copied(u));
            }
          } else {  // several small pages: a lane a copy
            const int b = lane / kCopyChunks, c = lane % kCopyChunks;
            __syncwarp();
            if (b < live)
              tma_load4(dst + c * kCopyStep + b * p.box * kCopyRow, val ? &vmap : &kmap, c * kCopyCols, 0,
                        head, id, copied(u));
          }
        }
        before += 2 * n;
      }
    } else if (warp == kLoadWarp) {
      // rows copied one by one, 16 bytes a lane: lane's addresses are those of rows
      // lane and lane + 32
      int issued = 0;
      constexpr int kElems = CODES ? 16 : 8, kPieces = DP / kElems;  // of 16 bytes
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
          const uint32_t dst = ring_addr + u * L::kUnitBytes + kCopyAt;
#pragma unroll
          for (int k = 0; k < 2; ++k)
            for (int i = 0; i < kPieces; ++i) {
              const int row = i * 32 / kPieces + lane / kPieces, j = lane % kPieces;
              const char* src = reinterpret_cast<const char*>(
                  __shfl_sync(~0u, reinterpret_cast<unsigned long long>(at[k]), row));
              const int rr = k * 32 + row;
              const bool on = src != nullptr && j * kElems < a.dim;
              // rows of 64 codes are not swizzled
              const int at16 = kCopyRow == 64 ? j : (j & 7) ^ (rr & 7);
              cp_async16(dst + (kCopyRow == 64 ? 0 : j / 8) * kCopyStep + rr * kCopyRow + (at16 << 4),
                         on ? src + j * 16 : a.k, on ? 16 : 0);
            }
          cp_async_commit();
          // the unit before the last has landed: hand it over
          if (issued >= 2) {
            cp_async_wait<2>();
            fence_async_smem();
            mbar_arrive(copied((issued - 2) % L::kUnits));
          }
        }
      }
      if (issued >= 2) {
        cp_async_wait<1>();
        fence_async_smem();
        mbar_arrive(copied((issued - 2) % L::kUnits));
      }
      cp_async_wait<0>();
      fence_async_smem();
      mbar_arrive(copied((issued - 1) % L::kUnits));
    }
    if (err != 0 && a.dev_error != nullptr) atomicOr(a.dev_error, static_cast<int32_t>(err));
  } else if (warp >= kMmaWarp && warp < kTurnWarp) {
    // ---------------------------------------------------------- products
    // One warp a stream: a wait takes some 150 cycles even where the phase is
    // over, and one warp for both streams spent more time in waits and issue than
    // the products take.  The whole warp walks, one lane issues.  What the
    // instructions' operands are formed from is the same in all lanes, and
    // shuffles say so to the compiler, which then keeps it in uniform registers:
    // operands moved there one by one took 80 cycles an instruction, against 48
    // (Q K^T, bound by reading Q and K from shared memory) and 64 (P V) of the
    // products themselves.
    constexpr uint32_t kQk = mma_idesc(kTile, false, CODES), kPv = mma_idesc(DP, true, CODES);
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
        if constexpr (CODES) mbar_arrive(smem_addr(&bars->s[s][b]));  // with what the turners wrote
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
  } else if (CODES && warp >= kTurnWarp) {
    // ---------------------------------------------------------- codes
    if constexpr (CODES)
      turn_codes<NS, DP, kTurners>(p, walk, warp - kTurnWarp, lane, ring, bars, copied, full, empty,
                                   timed_out);
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
    int cta_tiles = 0, qe = 0;  // of codes: tiles of the segments so far; the row's power of two
    WarpWalk<MR, EXT>* const ww = walks + warp;
    uint32_t tiles = 0;  // the stream's tiles so far
    uint32_t idle = 0;   // parity of the next segment without rows here
    int u0 = 0;          // ring position of the segment's first unit, and its turn
    uint32_t turn0 = 0;
    // the walk's next segment, by lane 0, into shared memory (tile1 = -1: none)
    auto advance = [&]() {
      __syncwarp();
      if (lane == 0) {
        Walk<MR, EXT> w = ww->walk;
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
      const bool live = st * kRows < g.rows;         // the stream has rows
      const bool work = st * kRows + wrow < g.rows;  // the warp has rows
      cp_async_wait<0>();
      if constexpr (CODES) {
        __syncwarp();  // the row came by the other lanes' copies
        if (work)
          qe = query_to_fp16<DP>(qbuf + st * L::kQBytes + wrow * 128, lane,
                                 min(32, g.rows - st * kRows - wrow), a.scale2 < 0.0f);
      }
      fence_async_smem();
      mbar_arrive(smem_addr(&bars->q[st]));
      // of this row; of a tree's the place of its key
      const int pos = g.seq - g.l + a.by_group.of(g.m * MR + st * kRows + row);
      const int lo = TREE ? tree_lo(a, g, pos) : a.window > 0 ? max(0, pos - a.window + 1) : 0;
      // keys that every row of the item sees: [all_lo, all_hi)
      const int all_hi = g.seq - g.l + (TREE ? 0 : a.by_group.of(g.m * MR) + 1);
      const int all_lo = TREE ? tree_all_lo(a, g) : a.window > 0
          ? max(0, g.seq - g.l + a.by_group.of(g.m * MR + g.rows - 1) - a.window + 1) : 0;
      // the largest score; of codes r, and D
      float m = -kInf, shift = 0.0f, l = 0.0f;

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
          constexpr uint32_t kOdd = CODES ? 0x7c00u : 0x7f80u;  // exponent of what is not finite
          if ((big & kOdd) == kOdd || (big & kOdd << 16) == kOdd << 16) {
            for (int at = row; at < L::kUnitBytes / 16; at += 128) {
              const int t = t0 + (at >> 3) % kTile;
              if (t >= all_lo && t < all_hi) continue;
              uint4 v = *reinterpret_cast<const uint4*>(unit + at * 16);
              uint32_t* w = reinterpret_cast<uint32_t*>(&v);
              bool odd = false;
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                if ((w[e] & kOdd) == kOdd) w[e] &= 0xffff0000u, odd = true;
                if ((w[e] & kOdd << 16) == kOdd << 16) w[e] &= 0xffffu, odd = true;
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
        if (CODES && work) {
          const uint32_t s_buf = s_at + buf * kTile;
          uint64_t bits = ~uint64_t{0};  // keys that the row sees
          if (edge) {
            if constexpr (TREE) {
              // a request of no length has no key, and rows behind the item's have no mask
              bits = g.seq > 0 && st * kRows + row < g.rows ? tree_bits(a, g, pos, lo, t0) : 0;
            } else {
              const int n = pos + 1 - t0;
              if (n < 64) bits = n > 0 ? (uint64_t{1} << n) - 1 : 0;
              if (lo > t0) bits &= lo - t0 < 64 ? ~uint64_t{0} << (lo - t0) : 0;
            }
          }
          float s[kTile];
          tmem_ld32(s_buf, reinterpret_cast<uint32_t*>(s));
          tmem_ld32(s_buf + 32, reinterpret_cast<uint32_t*>(s + 32));
          tmem_wait_ld();
          if (edge) {
            const uint32_t low = static_cast<uint32_t>(bits), high = static_cast<uint32_t>(bits >> 32);
#pragma unroll
            for (int k = 0; k < 32; ++k) {
              s[k] = low >> k & 1 ? s[k] : -kInf;
              s[k + 32] = high >> k & 1 ? s[k + 32] : -kInf;
            }
          }
          float mx[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
          for (int k = 4; k < kTile; k += 8)
#pragma unroll
            for (int e = 0; e < 4 && k + 2 * e < kTile; ++e) mx[e] = fmaxf(fmaxf(mx[e], s[k + 2 * e]), s[k + 2 * e + 1]);
          const int slot = (cta_tiles + tile - g.tile0) & 7, unit = qe + bars->key_exp[slot];  // of the scores
          const float top = scaled(fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])), unit);
          const float ct = fminf(fmaxf(scaled(c, unit), 0x1p-149f), FLT_MAX);
          const float e = bars->value_exp[slot];
          bool apart = false;  // weights far below one
          if (tile == g.tile0) {
            m = top, shift = e - kLift;
          } else {
            // log2 of the tile's largest above r, and of its weight above 2^7 (NaN, and no
            // rise, where neither it nor the tiles before have a key)
            const float above = (top - m) * c, most = above + (e - kLift) - shift;
            const bool rise = most > kRescale, raise = rise || above > kRaise;
            if (__any_sync(~0u, raise)) {
              const float up = raise && top > m ? above : 0.0f;
              const float now = rise ? (top > m ? 0.0f : above) + (e - kLift) : shift - up;
              const float f = rise ? ex2(shift - up - now) : 1.0f;
              l *= ex2(-up);
              m = raise ? fmaxf(m, top) : m, shift = now;
              if (__any_sync(~0u, rise)) {
                wait_o(tiles - 1);
#pragma unroll 1
                for (int k = 0; k < DP; k += 16) {
                  uint32_t o[16];
                  tmem_ld16(o_at + k, o);
                  tmem_wait_ld();
#pragma unroll
                  for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
                  tmem_st16(o_at + k, o);
                }
              }
            }
            apart = most < -kApart && top > -kInf;
          }
          const float ref = m == -kInf ? 0.0f : m;
          if (!__any_sync(~0u, apart || fabsf(ref * c) > kLargeScore)) {
            const float base = fmaf(ref, c, shift - e);
            const uint64_t mul2 = pack2(ct, ct), base2 = pack2(-base, -base);
            uint64_t sum[2] = {0, 0};
#pragma unroll
            for (int k = 0; k < kTile; k += 32) {
              uint32_t w[16];
#pragma unroll
              for (int i = 0; i < 16; ++i) {
                float p0, p1;
                unpack2(fma2(pack2(s[k + 2 * i], s[k + 2 * i + 1]), mul2, base2), &p0, &p1);
                p0 = ex2(p0), p1 = ex2(p1);
                sum[i & 1] = add2(sum[i & 1], pack2(p0, p1));
                asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(w[i]) : "f"(p1), "f"(p0));
              }
              tmem_st16(s_buf + k / 2, w);
            }
            float s0, s1;
            unpack2(add2(sum[0], sum[1]), &s0, &s1);
            // at most 2^113, but for a row that sees nothing of the tile: 0, not 0 times infinity
            l += (s0 + s1) * ex2(fminf(shift - e, 126.0f));
          } else {
            // scores so large that the rounding of r c would neither cancel nor be the same
            // beside each tile's E: differences of products first, exact where they count; or
            // weights so small that their part of l is a sum of its own.  S is read again, in a
            // short loop: the other tiles' instructions barely fit the cache (unrolled: chunks
            // 840 us for 760)
            const float u0 = pow2(unit >> 1), u1 = pow2(unit - (unit >> 1));
#pragma unroll 1
            for (int k = 0; k < kTile; k += 4) {
              uint32_t x[4], w[2];
              tmem_ld4(s_buf + k, x);
              tmem_wait_ld();
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                float y = __uint_as_float(x[i]);
                y = bits >> (k + i) & 1 ? (y * u0 * u1 - ref) * c : -kInf;
                l += ex2(y);
                x[i] = __float_as_uint(ex2(y - (shift - e)));
              }
#pragma unroll
              for (int i = 0; i < 2; ++i)
                asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(w[i]) : "f"(__uint_as_float(x[2 * i + 1])), "f"(__uint_as_float(x[2 * i])));
              tmem_st2(s_buf + k / 2, w);
            }
          }
          tmem_wait_st();
        }
        if (!CODES && work) {
          uint32_t x[kTile];
          tmem_ld32(s_at + buf * kTile, x);
          tmem_ld32(s_at + buf * kTile + 32, x + 32);
          tmem_wait_ld();
          float* s = reinterpret_cast<float*>(x);
          if (a.scale2 < 0.0f) {
#pragma unroll
            for (int k = 0; k < kTile; ++k) s[k] = -s[k];
          }
          if (TREE && edge) {
            // a request of no length has no key, and rows behind the item's have no mask
            const uint64_t bits = g.seq > 0 && st * kRows + row < g.rows ? tree_bits(a, g, pos, lo, t0) : 0;
            const uint32_t low = static_cast<uint32_t>(bits), high = static_cast<uint32_t>(bits >> 32);
#pragma unroll
            for (int k = 0; k < 32; ++k) {
              s[k] = low >> k & 1 ? s[k] : -kInf;
              s[k + 32] = high >> k & 1 ? s[k + 32] : -kInf;
            }
          }
          if (!TREE && edge) {
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
      cta_tiles += g.tile1 - g.tile0;
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
          float inv = g.whole || CODES ? (l > 0.0f || l != l ? 1.0f / l : 0.0f) : 1.0f;
          if (CODES) inv *= ex2(shift);
          const int prow = st * kRows + row;
          // rolled where segments are short: unrolled, its instructions come from far away
#pragma unroll (CODES ? 1 : DP / 64)
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
                if (TREE && !tree_sees(a, g, pos, t)) continue;
                const int page = a.by_page.of(t);
                int id = a.table[g.r * a.table_stride + page];
                if (id < 0 || id >= a.num_blocks) id = 0;
                const char* at = a.v + id * a.block + (t - page * a.page) * a.token + g.h * a.head;
                if constexpr (CODES) {  // NaN alone
#pragma unroll
                  for (int e = 0; e < 64; ++e)
                    if (k0 + e < a.dim && (at[k0 + e] & 0x7f) == 0x7f) o[e] = __uint_as_float(0x7fffffffu);
                } else {
                  const __nv_bfloat16* v = reinterpret_cast<const __nv_bfloat16*>(at) + k0;
#pragma unroll
                  for (int e = 0; e < 64; ++e)
                    if (k0 + e < a.dim && !(fabsf(__bfloat162float(v[e])) < kInf))
                      o[e] += __bfloat162float(v[e]);
                }
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
                    CODES ? make_float4(o[e] * inv, o[e + 1] * inv, o[e + 2] * inv, o[e + 3] * inv)
                          : make_float4(o[e], o[e + 1], o[e + 2], o[e + 3]);
            }
          }
          if (valid) {
            const float mc = m == -kInf ? -kInf : m * c;
            if (!g.whole)
              p.ml[static_cast<int64_t>(slot) * MR + prow] = make_float2(CODES ? m : mc, l);
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
        mbar_wait(copied(at % L::kUnits), (at / L::kUnits) & 1, late);
      }
    if (warp >= kMmaWarp && warp < kTurnWarp && done > 0)
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
// 2^(m c - max) (of codes, whose parts are means, times l over the sum of those) go to
// shared memory, then GROUPS threads sum four columns of a row, each over every GROUPS-th
// part, in worker order.  Bound by the latency of two rounds of loads,
// and by the partials' bytes (from L2) where there are many.
constexpr int kCombineRows = 4;

// threads of a group: four rows of DP / 4 columns, a whole number of warps per row
__host__ __device__ constexpr int combine_group(int dp) { return dp < 128 ? 128 : dp; }

template <int MR, int DP, int GROUPS, bool F32, bool CODES>
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
  const float c = CODES ? fabsf(a.scale2) : 1.0f;
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
        const float f = ex2(CODES ? (x.x - top) * c : x.x - top);
        weight[warp][i] = CODES ? x.y * f : f;
        l += x.y * f;
      }
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) l += __shfl_xor_sync(~0u, l, d);
      const float inv = l > 0.0f || l != l ? 1.0f / l : 0.0f;
      if (CODES) {  // before the sum: the parts may be as large as fp32 holds
        top *= c;
        for (int i = lane; i < r.parts; i += 32) weight[warp][i] *= inv;
      }
      if (lane == 0) {
        inverse[warp] = CODES ? 1.0f : inv;
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
