// sv_sample.cu -- one token per row with per-row temperature, top-k, top-p and
// min-p from given random numbers (include/spec_verify_serve.h).
//
// A cluster of C CTAs owns a row and streams it from HBM once.  It keeps, for
// every group of G 16-byte vectors (at most 512 bytes), the largest logit and,
// where the row's mass is needed, the group's mass relative to it, both in
// shared memory of rank 0, which then decides alone.  The kept set is a prefix of
// the order (value desc, id asc), so its last token (value t, id) describes it;
// min-p is a bar on the weight itself.
//  - No filter: the masses pick the group, one group is read again (from L2).
//  - Filters: at least R tokens are at or above the R-th largest group maximum.
//    With R = top_k, or 192 for top-p alone, only the groups that reach this bar
//    are read again, and their tokens at or above it make a list.  If it holds
//    the top-k set, or top_p of the mass, the row is finished on it: ranks by
//    counting, the cuts, the draw.  This is the path of usual rows.
//  - Otherwise (flat rows under top-p, top_k of hundreds) all CTAs of the row count
//    its tokens by weight in bins, collect the bin that the cut falls in and rank
//    its tokens.  Then one pass forms the groups' kept masses, and the draw is as
//    without filters.
//  - A bin too full for a list (many ties, as in bf16) is searched: an interval of
//    values around the cut is narrowed, three pivots a pass over the row, placed at
//    the bin's edges and then by interpolation, until it holds at most kCollect
//    tokens, which are collected and ranked, or one value, whose tokens are taken
//    by ascending id.
// A pass over the row after the first reads it from L2 and ends with an exchange:
// each CTA stores its partial into every CTA's shared memory, and after the cluster
// barrier all sum the C partials in rank order, so all decide alike.
//
// What bounds it.  One row: latency (151,936 bf16 under top-k 20 and top-p 0.95
// 8.4 us: 1.3 us to the settings, 1.3 us for the row on eight SMs, 0.9 us of
// cluster barriers, 3.5 us to decide).  Many rows: the stream at two CTAs an SM with
// the decision's latency between, and 512 rows are 1.7 times what fits (512 rows of
// 262,144 bf16, 268 MB: 65 us, 4.1 TB/s, 0.62 of the measured copy rate; four CTAs of
// 256 threads an SM 61 us, but 32 rows with their own settings took twice the time).
// Rows whose cut needs the bins: instructions, four passes over the row (96 flat
// fp32 rows of 129,280 under top-p 82 us), and at 64 registers a thread cut_by_bins and
// search spill some 300 bytes each.  Masked rows under top-k with fewer unmasked
// tokens than k: no bin holds the cut, and the search walks the keys down to -inf (10 of
// 151,936 bf16 under top-k 20: 84 us, where an unmasked row takes 9).
// Rows held in the cluster's shared memory instead of read again measured slower:
// 180 us for the 512 rows where reading again took 86, the resident bytes waiting
// through every decision.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "sv_host.cuh"
#include "sv_ptx.cuh"

namespace sv {
namespace serve {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;
constexpr int kList = 512;      // most tokens of a list
constexpr int kCollect = 512;   // most tokens that a search collects
constexpr int kBins = 2048;     // of 1/64 binade of weight
constexpr int kTopPSeeds = 192;  // group maxima that a top-p row's bar lies below
constexpr float kInf = __builtin_huge_valf();

struct SampleArgs {
  const char* logits;
  int64_t row_bytes;
  int32_t V, C, slice, shift;  // CTAs a row, vectors a slice, log2 vectors a group
  const float* temperature;
  const int32_t* top_k;
  const float *top_p, *min_p, *uniforms;
  int32_t* out_tokens;
  float* out_probs;
  int32_t* dev_error;
};

struct Header {
  float4 slot[2][kMaxCluster][2];  // exchanged partials, two exchanges in turn
  float4 part[kWarps][2];
  union {
    struct {
      uint64_t all[kList];  // rank 0: the list; key above complemented id
      float w[kList];       // rank 0: weights and ids, best first
      int32_t id[kList];
    };
    uint32_t bins[kBins];  // tokens by weight
  };
  uint64_t list[kCollect];  // this CTA's part of what a search collects
  uint64_t sum[kWarps];
  int32_t count, pick, cut, group, groups;
  float kept, total, base;
};
constexpr int kHeaderBytes = (sizeof(Header) + 127) / 128 * 128;

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::
                   : "memory");
}
__device__ __forceinline__ void store_peer(uint32_t addr, uint32_t rank, float4 v) {
  uint32_t peer;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(peer) : "r"(addr), "r"(rank));
  asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(peer), "f"(v.x), "f"(v.y),
               "f"(v.z), "f"(v.w)
               : "memory");
}

// Order-preserving key of a logit: 16 bits for bf16, 32 for fp32 (-0 below +0;
// values are compared as floats, where both are one).
template <int ES>
__device__ __forceinline__ uint32_t key_of(float x) {
  const uint32_t b = __float_as_uint(x);
  return (b ^ ((b >> 31) != 0 ? 0xffffffffu : 0x80000000u)) >> (ES == 2 ? 16 : 0);
}
template <int ES>
__device__ __forceinline__ float float_of(uint32_t k) {
  if constexpr (ES == 2) return __uint_as_float(((k >> 15) != 0 ? k ^ 0x8000u : ~k) << 16);
  return __uint_as_float((k >> 31) != 0 ? k ^ 0x80000000u : ~k);
}

template <int ES>
struct Vec {  // 16 bytes of logits
  static constexpr int N = 16 / ES;
  float x[N];
  __device__ __forceinline__ explicit Vec(const uint4& v) {
    if constexpr (ES == 2) {
      x[0] = bf16lo(v.x), x[1] = bf16hi(v.x), x[2] = bf16lo(v.y), x[3] = bf16hi(v.y);
      x[4] = bf16lo(v.z), x[5] = bf16hi(v.z), x[6] = bf16lo(v.w), x[7] = bf16hi(v.w);
    } else {
      x[0] = __uint_as_float(v.x), x[1] = __uint_as_float(v.y);
      x[2] = __uint_as_float(v.z), x[3] = __uint_as_float(v.w);
    }
  }
};

// A token's weight relative to the best one's: at most 1, and 1 for the best
// itself whatever the magnitude of the logits or the scale.
__device__ __forceinline__ float weight_of(float x, float best, float sc) {
  return ex2((x - best) * sc);
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(~0u, v, d);
  return v;
}
// Four vectors' values of a lane reduced over groups of 8 lanes: at each exchange a
// lane hands over half of what it has, so it ends with the result of vector
// folded(lane), after four exchanges for all; one by one they take twelve.
__device__ __forceinline__ int folded(int lane) { return (lane & 1) * 2 + (lane >> 1 & 1); }
template <typename Op>
__device__ __forceinline__ float fold(const float* v, Op op) {
  const bool odd = threadIdx.x & 1, second = threadIdx.x & 2;
  const float p = __shfl_xor_sync(~0u, odd ? v[0] : v[2], 1);
  const float q = __shfl_xor_sync(~0u, odd ? v[1] : v[3], 1);
  const float a = op(odd ? v[2] : v[0], p), b = op(odd ? v[3] : v[1], q);
  const float c = op(second ? b : a, __shfl_xor_sync(~0u, second ? a : b, 2));
  return op(c, __shfl_xor_sync(~0u, c, 4));
}
// A token in a list: larger is better (value desc, id asc; zeros alike).
__device__ __forceinline__ uint64_t entry_of(float x, int id) {
  const uint32_t b = __float_as_uint(x + 0.0f);
  const uint32_t k = b ^ ((b >> 31) != 0 ? 0xffffffffu : 0x80000000u);
  return static_cast<uint64_t>(k) << 32 | static_cast<uint32_t>(~id);
}
__device__ __forceinline__ float value_of(uint64_t e) {
  return float_of<4>(static_cast<uint32_t>(e >> 32));
}
__device__ __forceinline__ int id_of(uint64_t e) { return static_cast<int>(~static_cast<uint32_t>(e)); }

__device__ __forceinline__ uint32_t peer_addr(const void* p, int rank) {
  uint32_t peer;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(peer) : "r"(smem_addr(p)), "r"(rank));
  return peer;
}

template <int ES>
struct Row {
  static constexpr int N = 16 / ES;
  Header* h;
  float2* stat;          // rank 0: (largest logit, mass) of every group
  const char* base;      // the row, from the 16-byte boundary at or below it
  int lead, nvec;        // elements before the row in vector 0; its vectors
  int v0, v1;            // this CTA's vectors
  int V, G, C, rank, parity = 0;
  float best, sc;        // the row's maximum, log2(e) / T

  // Vector i; what the first and last hold beside the row is -inf.
  __device__ __forceinline__ uint4 load(int i) const {
    const char* p = base + static_cast<int64_t>(i) * 16;
    if (i * N >= lead && (i + 1) * N <= lead + V) return __ldg(reinterpret_cast<const uint4*>(p));
    union {
      uint4 v;
      uint16_t s[8];
      float f[4];
    } x;
#pragma unroll
    for (int e = 0; e < N; ++e) {
      const int id = i * N + e - lead;
      const bool in = id >= 0 && id < V;
      if constexpr (ES == 2) x.s[e] = in ? reinterpret_cast<const uint16_t*>(p)[e] : 0xff80u;
      else x.f[e] = in ? reinterpret_cast<const float*>(p)[e] : -kInf;
    }
    return x.v;
  }

  // Vectors i0 + lane, i0 + kThreads + lane, .. of this CTA's slice.  Whole
  // vectors of the row are loaded without a branch; its first and last one and
  // what lies past the slice (-inf) are put right after.
  static constexpr int kLoads = 4;
  __device__ __forceinline__ bool whole(int i0) const {  // nothing to put right
    return i0 >= (lead > 0 ? 1 : 0) &&
           i0 + (kLoads - 1) * kThreads + 32 <= min((lead + V) / N, v1);
  }
  __device__ __forceinline__ void fetch(int i0, uint4* x) const {
    const int in0 = lead > 0 ? 1 : 0, in1 = (lead + V) / N, i = i0 + (threadIdx.x & 31);
    const uint4* p = reinterpret_cast<const uint4*>(base);
    const uint32_t pad = ES == 2 ? 0xff80ff80u : 0xff800000u;
    if (whole(i0)) {
#pragma unroll
      for (int k = 0; k < kLoads; ++k) x[k] = __ldg(p + i + k * kThreads);
      return;
    }
    if (in1 > in0) {
#pragma unroll
      for (int k = 0; k < kLoads; ++k)
        x[k] = __ldg(p + max(min(i + k * kThreads, min(in1, v1) - 1), in0));
    }
#pragma unroll
    for (int k = 0; k < kLoads; ++k) {
      const int j = i + k * kThreads;
      if (j >= v1) x[k] = make_uint4(pad, pad, pad, pad);
      else if (j < in0 || j >= in1) x[k] = load(j);
    }
  }
  __device__ __forceinline__ int start() const { return v0 + (threadIdx.x >> 5) * 32; }

  // f(vector index, vector) over this CTA's vectors: a warp 32 together; every
  // lane takes part in every call.
  template <typename F>
  __device__ __forceinline__ void each(F f) const {
    for (int i0 = start(); i0 < v1; i0 += kThreads * kLoads) {
      uint4 x[kLoads];
      fetch(i0, x);
#pragma unroll
      for (int k = 0; k < kLoads; ++k)
        if (i0 + k * kThreads < v1) f(i0 + k * kThreads + static_cast<int>(threadIdx.x & 31), x[k]);
    }
  }

  __device__ __forceinline__ int token(int vec, int e) const { return vec * N + e - lead; }

  // Every CTA's partial, in rank order, to every thread.
  __device__ __forceinline__ const float4 (*exchange(float4 a, float4 b))[2] {
    if (threadIdx.x < C) {
      const uint32_t at = smem_addr(&h->slot[parity][rank][0]);
      store_peer(at, threadIdx.x, a);
      store_peer(at + 16, threadIdx.x, b);
    }
    cluster_sync();
    const float4(*s)[2] = h->slot[parity];
    parity ^= 1;
    return s;
  }

  // The threads' partials summed over warps, the CTA in warp order, and the row
  // in rank order.
  struct Sums {
    float m[3];
    int c[3];
  };
  __device__ __forceinline__ Sums total(Sums v) {
#pragma unroll
    for (int i = 0; i < 3; ++i) v.m[i] = warp_sum(v.m[i]), v.c[i] = __reduce_add_sync(~0u, v.c[i]);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) {
      h->part[threadIdx.x >> 5][0] = make_float4(v.m[0], v.m[1], v.m[2], 0);
      h->part[threadIdx.x >> 5][1] =
          make_float4(__int_as_float(v.c[0]), __int_as_float(v.c[1]), __int_as_float(v.c[2]), 0);
    }
    __syncthreads();
    float4 a = make_float4(0, 0, 0, 0);
    int c0 = 0, c1 = 0, c2 = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float4 x = h->part[w][0], y = h->part[w][1];
      a.x += x.x, a.y += x.y, a.z += x.z;
      c0 += __float_as_int(y.x), c1 += __float_as_int(y.y), c2 += __float_as_int(y.z);
    }
    const float4(*s)[2] = exchange(
        a, make_float4(__int_as_float(c0), __int_as_float(c1), __int_as_float(c2), 0));
    Sums r{{0, 0, 0}, {0, 0, 0}};
    for (int i = 0; i < C; ++i) {
      r.m[0] += s[i][0].x, r.m[1] += s[i][0].y, r.m[2] += s[i][0].z;
      r.c[0] += __float_as_int(s[i][1].x), r.c[1] += __float_as_int(s[i][1].y);
      r.c[2] += __float_as_int(s[i][1].z);
    }
    return r;
  }

  __device__ __forceinline__ float weight(float x) const { return weight_of(x, best, sc); }

  // Mass and count of the tokens at or above each of three values.
  __device__ __forceinline__ Sums at_least(const float t[3]) {
    Sums v{{0, 0, 0}, {0, 0, 0}};
    const float low = fminf(t[0], fminf(t[1], t[2]));
    each([&](int, const uint4& raw) {
      const Vec<ES> x(raw);
#pragma unroll
      for (int e = 0; e < N; ++e)
        if (x.x[e] >= low) {
          const float w = weight(x.x[e]);
#pragma unroll
          for (int j = 0; j < 3; ++j) {
            const bool on = x.x[e] >= t[j];
            v.m[j] += on ? w : 0.0f, v.c[j] += on ? 1 : 0;
          }
        }
    });
    return total(v);
  }

  // Into this CTA's list.
  __device__ __forceinline__ void append(float x, int id) {
    const int at = atomicAdd(&h->count, 1);
    if (at < kCollect) h->list[at] = entry_of(x, id);
  }
  // This CTA's list behind those of the ranks before it in rank 0's (`before`
  // tokens).
  __device__ __forceinline__ void send(int before) {
    const int n = h->count;
    const uint32_t peer = peer_addr(h->all, 0);
    for (int i = threadIdx.x; i < n; i += kThreads)
      asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(peer + (before + i) * 8), "l"(h->list[i])
                   : "memory");
    cluster_sync();
  }

  // Rank 0: weights and ids of the n listed tokens, best first.
  __device__ __forceinline__ void rank_list(int n) {
    if (threadIdx.x < 4 && n + threadIdx.x < kList) h->all[n + threadIdx.x] = 0;  // below any token
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += kThreads) {
      const uint64_t e = h->all[i];
      int r = 0;
      const ulonglong2* all = reinterpret_cast<const ulonglong2*>(h->all);
#pragma unroll 2
      for (int j = 0; j < n; j += 4) {
        const ulonglong2 x = all[j / 2], y = all[j / 2 + 1];
        r += (x.x > e ? 1 : 0) + (x.y > e ? 1 : 0) + (y.x > e ? 1 : 0) + (y.y > e ? 1 : 0);
      }
      h->w[r] = weight(value_of(e));
      h->id[r] = id_of(e);
    }
    __syncthreads();
  }

  // A warp of rank 0, over the ranked list: the first index (from 1) whose
  // running sum of weights reaches `need`, n if none does; *sum gets the sum
  // up to there.
  __device__ __forceinline__ int reach(int n, float need, float* sum) {
    const int lane = threadIdx.x & 31;
    float carry = 0;
    for (int base = 0; base < n; base += 32) {
      const int i = base + lane;
      float c = i < n ? h->w[i] : 0.0f;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const float o = __shfl_up_sync(~0u, c, d);
        if (lane >= d) c += o;
      }
      c += carry;
      const unsigned hit = __ballot_sync(~0u, i < n && c >= need);
      if (hit != 0) {
        const int l = __ffs(hit) - 1;
        *sum = __shfl_sync(~0u, c, l);
        return base + l + 1;
      }
      carry = __shfl_sync(~0u, c, min(31, n - 1 - base));
    }
    *sum = carry;
    return n;
  }
};

// The last kept token of a cut, and the mass of what it keeps.
struct Cut {
  float t;
  int id;
  float mass;
  int parity = 0;   // of the row's next exchange
  bool ok = true;
  float lo = kInf, hi = -kInf;  // not ok: values that the cut probably lies between, if lo <= hi
};

// The cut at the k-th best token (need < 0), or where the mass reaches `need`,
// among the tokens up to `within`: the tokens below top_x counted by 1/64 binade
// of weight (one pass; each counts as its weight relative to the bin's middle, in
// whole 2^-12; with plain counts one row in ten missed the bin and took the search:
// 96 flat rows of 151,936 bf16 132 us, 80 now), the bins around the cut collected and
// ranked (another).
// Tokens at or above top_x (infinite: none) number c_top, with mass m_top; the
// cut does not lie below floor_x.  The
// bins' masses are estimates, the masses that decide
// are sums; not ok if the cut lies outside what was collected.
template <int ES>
__device__ __noinline__ Cut cut_by_bins(Row<ES> R, int k, float need, Cut within, float top_x,
                                        float m_top, int c_top, float floor_x) {
  constexpr int N = 16 / ES, kPer = kBins / kThreads;
  constexpr uint32_t kUnit = 4096;             // a token of its bin's middle weight
  constexpr float kSlope = 0.01083042469625f;  // log(2) / 64: a bin's width in the weights
  static_assert(SV_SAMPLE_MAX_ROW_BYTES / 2 * (kUnit * 1.006) < 4294967295.0, "a bin's sum");
  const bool by_mass = need >= 0.0f;
  Header* h = R.h;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const float origin = top_x < kInf ? top_x : R.best, step = fminf(R.sc * 64.0f, 3.0e38f);
  // rounded to the nearest by an addition (conversions run at a quarter of its rate)
  auto bin_at = [&](float x) { return fminf((origin - x) * step, kBins - 1.0f); };
  auto bin_of = [&](float x) {
    return __float_as_int(bin_at(x) + 0x1p23f) - __float_as_int(0x1p23f);
  };
  const float low = fmaxf(fmaxf(floor_x, within.t), -3.4028235e38f);
  // of tokens at within.t only some may count; NaN: all do
  const float tie = within.id != INT32_MAX ? within.t : __int_as_float(0x7fc00000);
  auto inside = [&](float x, int id) {
    return (x < top_x) & (x >= low) && !(x == tie && id > within.id);
  };
  for (int i = tid; i < kBins; i += kThreads) h->bins[i] = 0;
  __syncthreads();
  R.each([&](int i, const uint4& raw) {
    const Vec<ES> x(raw);
#pragma unroll
    for (int e = 0; e < N; ++e)
      if (inside(x.x[e], R.token(i, e))) {
        const float y = bin_at(x.x[e]), near = y + 0x1p23f, off = y - (near - 0x1p23f);
        const uint32_t w = by_mass ? __float_as_uint(fmaf(off, -kSlope * kUnit, 0x1p23f + kUnit)) -
                                         __float_as_uint(0x1p23f)
                                   : kUnit;
        atomicAdd(&h->bins[__float_as_int(near) - __float_as_int(0x1p23f)], w);
      }
  });
  cluster_sync();
  int first = 0, end = 0, at_bin = 0;  // bins to collect; the cut's
  if (R.rank == 0) {
    static_assert(kPer == 4, "one 16-byte load a thread and rank");
    uint4 x[kMaxCluster];
#pragma unroll
    for (int r = 0; r < kMaxCluster; ++r)
      if (r < R.C)
        asm volatile("ld.shared::cluster.v4.u32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(x[r].x), "=r"(x[r].y), "=r"(x[r].z), "=r"(x[r].w)
                     : "r"(peer_addr(&h->bins[tid * kPer], r)));
    uint32_t units[kPer] = {0, 0, 0, 0};
#pragma unroll
    for (int r = 0; r < kMaxCluster; ++r)
      if (r < R.C)
        units[0] += x[r].x, units[1] += x[r].y, units[2] += x[r].z, units[3] += x[r].w;
    const float w0 = R.weight(origin) * (1.0f / kUnit);
    int n[kPer];
    float mass[kPer], m = 0;
    int c = 0;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      n[j] = static_cast<int>((units[j] + kUnit / 2) / kUnit);
      mass[j] = static_cast<float>(units[j]) * w0 * ex2(-(tid * kPer + j) / 64.0f);
      m += mass[j], c += n[j];
    }
    float mi = m;
    int ci = c;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const float om = __shfl_up_sync(~0u, mi, d);
      const int oc = __shfl_up_sync(~0u, ci, d);
      if (lane >= d) mi += om, ci += oc;
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kPer; ++j) h->bins[tid * kPer + j] = n[j];
    if (lane == 31) h->part[warp][0] = make_float4(mi, __int_as_float(ci), 0, 0);
    if (tid == 0) h->cut = kBins;
    __syncthreads();
    mi += m_top, ci += c_top;
    for (int w = 0; w < warp; ++w) mi += h->part[w][0].x, ci += __float_as_int(h->part[w][0].y);
    mi -= m, ci -= c;  // before this thread's bins
    int at = kBins;
    float past = 0.5f;  // how much of the bin lies past the cut
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      mi += mass[j], ci += n[j];
      if (n[j] > 0 && (by_mass ? mi >= need : ci >= k)) {
        at = tid * kPer + j;
        if (by_mass) past = (mi - need) / mass[j];
        break;
      }
    }
    if (at < kBins) atomicMin(&h->cut, at);
    __syncthreads();
    if (at < kBins && at == h->cut) h->base = past;
    __syncthreads();
    if (tid == 0) {  // the cut's bin and its neighbours, while a list holds them
      constexpr int kMost = kCollect - 4, kFew = kCollect / 2;  // counts are off by half a percent
      int b = h->cut, lo = b, hi = b + 1;
      int total = b < kBins - 1 ? static_cast<int>(h->bins[b]) : kCollect;
      auto fits = [&](int i, int most) {
        return i >= 0 && i < kBins - 1 && total + static_cast<int>(h->bins[i]) <= most;
      };
      // near an edge of the bin the cut may lie in the next
      if (h->base < 0.0625f && fits(hi, kMost)) total += h->bins[hi++];
      if (h->base > 0.9375f && fits(lo - 1, kMost)) total += h->bins[--lo];
      for (int j = 0; j < 4; ++j) {
        if (fits(hi, kFew)) total += h->bins[hi++];
        if (fits(lo - 1, kFew)) total += h->bins[--lo];
      }
      if (total > kMost) lo = hi = 0;
      h->group = lo, h->groups = hi;
    }
    __syncthreads();
    first = h->group, end = h->groups, at_bin = h->cut;
  }
  __syncthreads();
  if (tid == 0) h->count = 0;
  {
    const float4(*s)[2] = R.exchange(
        make_float4(__int_as_float(first), __int_as_float(end), __int_as_float(at_bin), 0),
        make_float4(0, 0, 0, 0));
    first = __float_as_int(s[0][0].x), end = __float_as_int(s[0][0].y);
    at_bin = __float_as_int(s[0][0].z);
  }
  Cut cut{0.0f, -1, 0.0f, R.parity, false};
  if (at_bin < kBins - 1) {  // for the search
    const float wide = end == 0 ? 0.5f : 3.0f;
    cut.lo = origin - (at_bin + wide) / step, cut.hi = origin - (at_bin - wide) / step;
  }
  if (end == 0) return cut;
  typename Row<ES>::Sums v{{0, 0, 0}, {0, 0, 0}};  // mass and count above the collected bins
  R.each([&](int i, const uint4& raw) {
    const Vec<ES> x(raw);
#pragma unroll
    for (int e = 0; e < N; ++e)
      if (inside(x.x[e], R.token(i, e))) {
        const int b = bin_of(x.x[e]);
        if (b < first) v.m[0] += R.weight(x.x[e]), ++v.c[0];
        else if (b < end) R.append(x.x[e], R.token(i, e));
      }
  });
  __syncthreads();
  v.c[1] = tid == 0 ? h->count : 0;
  const int turn = R.parity;
  const typename Row<ES>::Sums s = R.total(v);
  int before = 0;
  for (int r = 0; r < R.rank; ++r) before += __float_as_int(h->slot[turn][r][1].y);
  R.send(before);
  if (R.rank == 0) {
    const int n = s.c[1];
    const float above = m_top + s.m[0];
    R.rank_list(n);
    if (warp == 0) {
      float sum;
      const int want = by_mass ? n : k - c_top - s.c[0];
      const int at = R.reach(min(n, max(want, 1)), by_mass ? need - above : kInf, &sum);
      // the cut is here if something of it was left, and there was enough
      const bool ok = by_mass ? need > above && above + sum >= need : want >= 1 && want <= n;
      if (lane == 0) h->pick = ok ? h->id[at - 1] : -1, h->kept = above + sum;
    }
    __syncthreads();
    for (int i = tid; i < n; i += kThreads)
      if (id_of(h->all[i]) == h->pick) h->total = value_of(h->all[i]);
    __syncthreads();
  }
  const float4(*f)[2] = R.exchange(make_float4(h->total, __int_as_float(h->pick), h->kept, 0),
                                   make_float4(0, 0, 0, 0));
  cut.t = f[0][0].x, cut.id = __float_as_int(f[0][0].y), cut.mass = f[0][0].z;
  cut.parity = R.parity, cut.ok = cut.id >= 0;
  return cut;
}

// The cut at the k-th best token (need < 0), or where the mass reaches `need`,
// within the tokens at or above key `lo` (of which ties at its value only up
// to id `lo_id`); f_lo >= target > 0 there.  above: a value with fewer than k
// tokens, or less mass than need, at or above it, their count and mass.
template <int ES>
__device__ __noinline__ Cut search(Row<ES> R, int k, float need, uint32_t lo, int lo_id,
                                   float m_lo, int c_lo, uint32_t hi, float m_hi, int c_hi,
                                   float guess_lo, float guess_hi) {
  const bool by_mass = need >= 0.0f;
  constexpr uint32_t kLow = ES == 2 ? 0x7fu : 0x7fffffu;  // key of -inf
  for (int iter = 0; hi - lo > 1 && c_lo - c_hi > kCollect; ++iter) {
    const float xh = fminf(float_of<ES>(hi), R.best), xl = float_of<ES>(lo);
    uint32_t p[3];
    if (iter == 0 && guess_lo <= guess_hi) {
      // a bin too full for a list; in bf16 often one value: the two keys around it
      p[0] = key_of<ES>(guess_lo), p[2] = key_of<ES>(guess_hi) + 1;
      if (float_of<ES>(p[0]) < guess_lo && p[0] + 1 < p[2]) ++p[0];
      p[1] = p[0] + (p[2] - p[0]) / 2;
    } else if (iter < 8 && lo == kLow) {  // no lower end yet: steps of some binades of weight
      const float unit = 1.0f / R.sc;
#pragma unroll
      for (int j = 0; j < 3; ++j)
        p[2 - j] = key_of<ES>(xh - (j == 0 ? 1.5f : j == 1 ? 3.0f : 6.0f) * unit);
    } else if (iter < 8) {  // around the interpolated cut
      const float f = by_mass ? (m_lo - need) / (m_lo - m_hi)
                              : static_cast<float>(c_lo - k) / static_cast<float>(c_lo - c_hi);
      const float at = xl + (xh - xl) * f, d = (xh - xl) * 0.04f;
      p[0] = key_of<ES>(at - d), p[1] = key_of<ES>(at), p[2] = key_of<ES>(at + d);
    } else {  // quarters of the keys
      const uint32_t q = (hi - lo) / 4;
      p[0] = lo + q, p[1] = lo + 2 * q, p[2] = lo + 3 * q;
    }
    float t[3];
#pragma unroll
    for (int j = 0; j < 3; ++j) {
      p[j] = min(max(p[j], lo + 1), hi - 1);
      t[j] = float_of<ES>(p[j]);
    }
    const typename Row<ES>::Sums s = R.at_least(t);
#pragma unroll
    for (int j = 0; j < 3; ++j) {  // pivots rise
      const bool reached = by_mass ? s.m[j] >= need : s.c[j] >= k;
      if (reached && p[j] >= lo) lo = p[j], m_lo = s.m[j], c_lo = s.c[j], lo_id = -1;
    }
#pragma unroll
    for (int j = 2; j >= 0; --j) {
      const bool reached = by_mass ? s.m[j] >= need : s.c[j] >= k;
      if (!reached && p[j] > lo && p[j] <= hi) hi = p[j], m_hi = s.m[j], c_hi = s.c[j];
    }
  }
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  Header* h = R.h;
  constexpr int N = 16 / ES;
  const float tl = float_of<ES>(lo), th = float_of<ES>(hi);
  const bool top = hi > key_of<ES>(R.best);  // nothing lies above
  Cut cut;
  if (c_lo - c_hi <= kCollect) {  // the few tokens of the interval, ranked
    __syncthreads();
    if (tid == 0) h->count = 0;
    __syncthreads();
    R.each([&](int i, const uint4& raw) {
      const Vec<ES> v(raw);
#pragma unroll
      for (int e = 0; e < N; ++e) {
        const int id = R.token(i, e);
        if ((v.x[e] >= tl) & (top | (v.x[e] < th)) & (id >= 0) & (id < R.V)) R.append(v.x[e], id);
      }
    });
    __syncthreads();
    const float4(*s)[2] = R.exchange(make_float4(__int_as_float(h->count), 0, 0, 0),
                                     make_float4(0, 0, 0, 0));
    int before = 0, n = 0;
    for (int r = 0; r < R.C; ++r) {
      if (r < R.rank) before += __float_as_int(s[r][0].x);
      n += __float_as_int(s[r][0].x);
    }
    R.send(before);
    if (R.rank == 0) {
      R.rank_list(n);
      if (warp == 0) {
        float sum;
        const int at = by_mass ? R.reach(n, need - m_hi, &sum)
                               : R.reach(min(n, k - c_hi), kInf, &sum);
        if (lane == 0) {
          // the value itself, from the entry with this id
          h->cut = at - 1;
          h->kept = m_hi + sum;
        }
      }
      __syncthreads();
      for (int i = tid; i < n; i += kThreads)
        if (id_of(h->all[i]) == h->id[h->cut]) h->total = value_of(h->all[i]);
      __syncthreads();
      cut.t = h->total, cut.id = h->id[h->cut], cut.mass = h->kept;
    }
    const float4(*f)[2] =
        R.exchange(make_float4(cut.t, __int_as_float(cut.id), cut.mass, 0), make_float4(0, 0, 0, 0));
    cut.t = f[0][0].x, cut.id = __float_as_int(f[0][0].y), cut.mass = f[0][0].z;
  } else {  // one value: the lowest ids of its class
    cut.t = tl;
    const float w = R.weight(cut.t);
    int64_t ties;
    if (by_mass) {
      const float more = w > 0.0f ? ceilf((need - m_hi) / w) : 1.0f;
      ties = static_cast<int64_t>(fminf(fmaxf(more, 1.0f), 2.0e9f));
    } else {
      ties = k - c_hi;
    }
    cut.mass = m_hi + static_cast<float>(ties) * w;
    // per warp's run of the CTA's vectors, so that ids ascend over runs and ranks
    const int run = (R.v1 - R.v0 + kWarps - 1) / kWarps;
    const int r0 = min(R.v1, R.v0 + warp * run), r1 = min(R.v1, r0 + run);
    int c = 0;
    for (int i = r0 + lane; i < r1; i += 32) {
      const Vec<ES> v(R.load(i));
#pragma unroll
      for (int e = 0; e < N; ++e) c += v.x[e] == cut.t ? 1 : 0;
    }
    const int mine = __reduce_add_sync(~0u, c);
    __syncthreads();
    if (tid == 0) h->pick = -1;
    if (lane == 0) h->part[warp][0].x = __int_as_float(mine);
    __syncthreads();
    int before = 0, cta = 0, all = 0;
    for (int w2 = 0; w2 < kWarps; ++w2) {
      if (w2 < warp) before += __float_as_int(h->part[w2][0].x);
      cta += __float_as_int(h->part[w2][0].x);
    }
    const float4(*s)[2] =
        R.exchange(make_float4(__int_as_float(cta), 0, 0, 0), make_float4(0, 0, 0, 0));
    for (int r = 0; r < R.C; ++r) {
      if (r < R.rank) before += __float_as_int(s[r][0].x);
      all += __float_as_int(s[r][0].x);
    }
    if (ties < all && before < ties && before + mine >= ties) {  // this warp's run holds it
      int left = static_cast<int>(ties) - before;
      for (int i0 = r0; i0 < r1; i0 += 32) {
        const int i = i0 + lane;
        int n = 0;
        if (i < r1) {
          const Vec<ES> v(R.load(i));
#pragma unroll
          for (int e = 0; e < N; ++e) n += v.x[e] == cut.t ? 1 : 0;
        }
        int inc = n;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
          const int o = __shfl_up_sync(~0u, inc, d);
          if (lane >= d) inc += o;
        }
        if (i < r1 && inc - n < left && inc >= left) {
          const Vec<ES> v(R.load(i));
          int seen = inc - n;
#pragma unroll
          for (int e = 0; e < N; ++e)
            if (v.x[e] == cut.t && ++seen == left) h->pick = R.token(i, e);
        }
        const int step = __shfl_sync(~0u, inc, 31);
        if (step >= left) break;
        left -= step;
      }
    }
    __syncthreads();
    const float4(*f)[2] =
        R.exchange(make_float4(__int_as_float(h->pick), 0, 0, 0), make_float4(0, 0, 0, 0));
    cut.id = INT32_MAX;
    if (ties < all)
      for (int r = 0; r < R.C; ++r)
        if (__float_as_int(f[r][0].x) >= 0) cut.id = __float_as_int(f[r][0].x);
  }
  if (lo_id >= 0 && cut.t == tl && cut.id > lo_id) cut.id = lo_id;
  cut.parity = R.parity;
  return cut;
}

// Rank 0: the token, from the groups' masses stat[].y (relative to the best
// token): the group that holds u * total, then its tokens.
template <int ES>
__device__ __forceinline__ void draw(Row<ES>& R, const SampleArgs& a, int row, int groups, float u,
                                     Cut cut, float min_p) {
  constexpr int N = 16 / ES;
  Header* h = R.h;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (groups + kThreads - 1) / kThreads;
  const int g0 = min(groups, tid * per), g1 = min(groups, g0 + per);
  float own = 0;
  for (int g = g0; g < g1; ++g) own += R.stat[g].y;
  float inc = own;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const float o = __shfl_up_sync(~0u, inc, d);
    if (lane >= d) inc += o;
  }
  __syncthreads();
  if (lane == 31) h->part[warp][0].x = inc;
  if (tid == 0) h->pick = INT32_MAX, h->cut = -1;
  __syncthreads();
  float before = 0, total = 0;
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) before += h->part[w][0].x;
    total += h->part[w][0].x;
  }
  const float target = u * total;
  float cum = before + (inc - own);
  if (own > 0.0f) {
    if (cum + own > target) atomicMin(&h->pick, tid);
    atomicMax(&h->cut, tid);
  }
  __syncthreads();
  if (tid == (h->pick != INT32_MAX ? h->pick : h->cut)) {
    int last = g0;
    float base = cum;
    for (int g = g0; g < g1; ++g) {
      const float m = R.stat[g].y;
      if (m > 0.0f) last = g, base = cum;
      cum += m;
      if (m > 0.0f && cum > target) break;
    }
    h->group = last, h->base = base;
  }
  __syncthreads();
  if (warp != 0) return;
  const int vec = h->group * R.G + lane;
  float w[N], k = 0;
#pragma unroll
  for (int e = 0; e < N; ++e) w[e] = 0;
  if (lane < R.G && vec < R.nvec) {
    const Vec<ES> v(R.load(vec));
#pragma unroll
    for (int e = 0; e < N; ++e) {
      const float x = v.x[e];
      if (x > cut.t || (x == cut.t && R.token(vec, e) <= cut.id)) w[e] = R.weight(x);
      if (w[e] < min_p) w[e] = 0.0f;
      k += w[e];
    }
  }
  inc = k;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const float o = __shfl_up_sync(~0u, inc, d);
    if (lane >= d) inc += o;
  }
  float c = h->base + (inc - k);
  int id = -1, last = -1;
  float iw = 0, lw = 0;
#pragma unroll
  for (int e = 0; e < N; ++e) {
    c += w[e];
    if (w[e] > 0.0f) {
      last = R.token(vec, e), lw = w[e];
      if (id < 0 && c > target) id = last, iw = w[e];
    }
  }
  const unsigned hit = __ballot_sync(~0u, id >= 0), any = __ballot_sync(~0u, last >= 0);
  // without a hit the sums' rounding left the target past the group: its last token
  const int from = hit != 0 ? __ffs(hit) - 1 : 31 - __clz(any);
  if (lane == from) {
    a.out_tokens[row] = hit != 0 ? id : last;
    if (a.out_probs != nullptr) a.out_probs[row] = (hit != 0 ? iw : lw) / total;
  }
}

// PER_SM: CTAs an SM that the registers are cut for.
template <int ES, int PER_SM>
__global__ __launch_bounds__(kThreads, PER_SM) void sample_kernel(const SampleArgs a) {
  extern __shared__ __align__(128) char smem[];
  constexpr int N = 16 / ES;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int row = blockIdx.x / a.C, rank = a.C > 1 ? static_cast<int>(cluster_rank()) : 0;
  Header* h = reinterpret_cast<Header*>(smem);
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");

  Row<ES> R;
  const char* src = a.logits + row * a.row_bytes;
  R.h = h, R.stat = reinterpret_cast<float2*>(smem + kHeaderBytes);
  R.lead = static_cast<int>(reinterpret_cast<uintptr_t>(src) & 15) / ES;
  R.base = src - R.lead * ES;
  R.V = a.V, R.G = 1 << a.shift, R.C = a.C, R.rank = rank;
  R.nvec = (R.lead + a.V + N - 1) / N;
  R.v0 = min(R.nvec, rank * a.slice), R.v1 = min(R.nvec, R.v0 + a.slice);
  const int G = R.G, groups = (R.nvec + G - 1) >> a.shift;

  // ---- the first loads are on their way while the settings arrive
  const int i_first = R.start();
  uint4 ahead[Row<ES>::kLoads];
  if (i_first < R.v1) R.fetch(i_first, ahead);

  // ---- the row's settings
  const float T = a.temperature != nullptr ? a.temperature[row] : 1.0f;
  int top_k = a.top_k != nullptr ? a.top_k[row] : 0;
  float top_p = a.top_p != nullptr ? a.top_p[row] : 1.0f;
  float min_p = a.min_p != nullptr ? a.min_p[row] : 0.0f;
  const float u = a.uniforms[row];
  uint32_t err = 0;
  if (!(T >= 0.0f && T < kInf) || !(top_p > 0.0f && top_p <= 1.0f) ||
      !(min_p >= 0.0f && min_p <= 1.0f) || !(u >= 0.0f && u < 1.0f))
    err = SV_DEVERR_PARAM;
  if (T == 0.0f) top_k = 1, top_p = 1.0f, min_p = 0.0f;  // the best token alone
  if (top_k >= a.V) top_k = 0;
  R.sc = T == 0.0f ? 1.0f : fminf(1.4426950408889634f / T, 3.0e38f);
  const bool use_k = top_k > 0, use_p = top_p < 1.0f, filtered = use_k || use_p || min_p > 0.0f;
  const bool need_mass = !use_k && (use_p || !filtered);
  if (tid == 0) h->count = 0, h->groups = 0;

  // ---- one pass: every group's largest logit (NaN wins) and mass
  bool joined = false;
  const uint32_t stat0 = peer_addr(R.stat, 0);
  auto join = [&] {  // every CTA of the row runs: rank 0's memory can be written
    if (!joined) {
      asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
      joined = true;
    }
  };
  auto group = [&](int i, const uint4& raw) {
    float m;
    if constexpr (ES == 2) {
      const uint32_t p = bf16x2_max_nan(bf16x2_max_nan(raw.x, raw.y), bf16x2_max_nan(raw.z, raw.w));
      m = fmax_nan(bf16lo(p), bf16hi(p));
    } else {
      const Vec<4> x(raw);
      m = fmax_nan(fmax_nan(x.x[0], x.x[1]), fmax_nan(x.x[2], x.x[3]));
    }
    for (int d = 1; d < G; d <<= 1) m = fmax_nan(m, __shfl_xor_sync(~0u, m, d));
    float s = 0;
    if (need_mass) {
      const Vec<ES> x(raw);
      const float ref = m == -kInf ? 0.0f : m;
#pragma unroll
      for (int e = 0; e < N; ++e) s += weight_of(x.x[e], ref, R.sc);
      for (int d = 1; d < G; d <<= 1) s += __shfl_xor_sync(~0u, s, d);
    }
    join();
    if ((lane & (G - 1)) == 0 && i < R.v1)
      asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(stat0 + (i >> a.shift) * 8),
                   "f"(m), "f"(s)
                   : "memory");
  };
  // the usual size, 8 vectors a group, four groups at once
  auto four = [&](int i0, const uint4* raw) {
    float v[4], m;
    if constexpr (ES == 2) {
#pragma unroll
      for (int k = 0; k < 4; ++k)
        v[k] = __uint_as_float(bf16x2_max_nan(bf16x2_max_nan(raw[k].x, raw[k].y),
                                              bf16x2_max_nan(raw[k].z, raw[k].w)));
      const uint32_t f = __float_as_uint(fold(v, [](float x, float y) {
        return __uint_as_float(bf16x2_max_nan(__float_as_uint(x), __float_as_uint(y)));
      }));
      m = fmax_nan(bf16lo(f), bf16hi(f));
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const Vec<4> x(raw[k]);
        v[k] = fmax_nan(fmax_nan(x.x[0], x.x[1]), fmax_nan(x.x[2], x.x[3]));
      }
      m = fold(v, [](float x, float y) { return fmax_nan(x, y); });
    }
    float s = 0;
    if (need_mass) {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float top = __shfl_sync(~0u, m, (lane & 24) | (k >> 1) | (k & 1) << 1);
        const float ref = top == -kInf ? 0.0f : top;
        const Vec<ES> x(raw[k]);
        v[k] = 0;
#pragma unroll
        for (int e = 0; e < N; ++e) v[k] += weight_of(x.x[e], ref, R.sc);
      }
      s = fold(v, [](float x, float y) { return x + y; });
    }
    join();
    const int i = i0 + folded(lane) * kThreads + (lane & 24);  // the group's first vector
    if ((lane & 4) == 0 && i < R.v1)
      asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(stat0 + i), "f"(m), "f"(s)
                   : "memory");
  };
  for (int i0 = i_first; i0 < R.v1; i0 += kThreads * Row<ES>::kLoads) {
    uint4 x[Row<ES>::kLoads];
#pragma unroll
    for (int k = 0; k < Row<ES>::kLoads; ++k) x[k] = ahead[k];
    if (i0 + kThreads * Row<ES>::kLoads < R.v1) R.fetch(i0 + kThreads * Row<ES>::kLoads, ahead);
    if (G == 8) {
      four(i0, x);
      continue;
    }
#pragma unroll
    for (int k = 0; k < Row<ES>::kLoads; ++k)
      if (i0 + k * kThreads < R.v1) group(i0 + k * kThreads + lane, x[k]);
  }
  if (!joined) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  cluster_sync();

  // ---- rank 0 decides
  float bar_x = -kInf, list_mass = 0.0f, row_mass = 0.0f;
  int listed = 0;
  bool more = false;
  if (rank == 0) {
    float mx = -kInf;
    for (int g = tid; g < groups; g += kThreads) mx = fmax_nan(mx, R.stat[g].x);
    const float own = mx;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) mx = fmax_nan(mx, __shfl_xor_sync(~0u, mx, d));
    if (lane == 0) h->part[warp][0].x = mx;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kWarps; ++w) mx = fmax_nan(mx, h->part[w][0].x);
    R.best = mx;
    if (!(mx > -kInf && mx < kInf)) err |= SV_DEVERR_NAN;
    if (err != 0) {
      if (tid == 0) {
        a.out_tokens[row] = -1;
        if (a.out_probs != nullptr) a.out_probs[row] = 0.0f;
        if (a.dev_error != nullptr) atomicOr(a.dev_error, static_cast<int32_t>(err));
      }
    } else {
      if (need_mass) {  // masses relative to the best token, and their sum
        float s = 0;
        for (int g = tid; g < groups; g += kThreads) {
          const float2 x = R.stat[g];
          const float m = x.x == -kInf ? 0.0f : x.y * R.weight(x.x);
          R.stat[g].y = m;
          s += m;
        }
        s = warp_sum(s);
        __syncthreads();
        if (lane == 0) h->part[warp][0].x = s;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < kWarps; ++w) row_mass += h->part[w][0].x;
      }
      if (!filtered) {
        draw<ES>(R, a, row, groups, u, Cut{-kInf, INT32_MAX, 0.0f}, 0.0f);
      } else {
        // -- the bar
        const int want = min(use_k ? top_k : kTopPSeeds, min(groups, kThreads));
        if (!use_k && !use_p) {  // min-p alone: its own bar, a little lower
          bar_x = fmaf(__log2f(min_p) - 0.001f, 1.0f / R.sc, mx) - fabsf(mx) * 1e-6f;
        } else if (want == 1 && use_k) {
          bar_x = mx;
        } else if (a.V > kList) {
          // the want-th largest of the threads' maxima over their groups, by the
          // upper 16 bits of the keys: the bar may be lower than it, not higher
          const uint32_t seed = key_of<4>(own) >> 16;
          uint32_t at = 0;
          for (uint32_t bit = 0x8000u; bit != 0; bit >>= 1)
            if (__syncthreads_count(seed >= (at | bit)) >= want) at |= bit;
          bar_x = at <= 0x7fu ? -kInf : float_of<4>(at << 16);
        }
        // -- the groups that reach it, and their tokens that do
        int32_t* reached = h->id;  // until the list is ranked
        __syncthreads();
        for (int g = tid; g < groups; g += kThreads)
          if (R.stat[g].x >= bar_x) {
            const int at = atomicAdd(&h->groups, 1);
            if (at < kList) reached[at] = g;
          }
        __syncthreads();
        const int vecs = min(h->groups, kList) << a.shift;
        uint64_t sum = 0;  // in 2^-40: the groups' order in the list changes nothing
        if (h->groups <= kList) {
          const int in0 = R.lead > 0 ? 1 : 0, in1 = (R.lead + a.V) / N;
          for (int i0 = tid; i0 < vecs; i0 += kThreads * 4) {
            uint4 x[4];
            int v[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const int i = i0 + k * kThreads;
              v[k] = i < vecs ? (reached[i >> a.shift] << a.shift) + (i & (G - 1)) : R.nvec;
            }
            if (in1 > in0) {  // whole vectors first, without a branch
#pragma unroll
              for (int k = 0; k < 4; ++k)
                x[k] = __ldg(reinterpret_cast<const uint4*>(R.base) + max(min(v[k], in1 - 1), in0));
            }
#pragma unroll
            for (int k = 0; k < 4; ++k)
              if (v[k] < R.nvec && (v[k] < in0 || v[k] >= in1)) x[k] = R.load(v[k]);
#pragma unroll
            for (int k = 0; k < 4; ++k)
              if (v[k] < R.nvec) {
                const Vec<ES> y(x[k]);
#pragma unroll
                for (int e = 0; e < N; ++e)
                  if (y.x[e] >= bar_x) {
                    sum += static_cast<uint64_t>(R.weight(y.x[e]) * 0x1p40f);
                    const int id = R.token(v[k], e);
                    if (id >= 0 && id < a.V) {
                      const int at = atomicAdd(&h->count, 1);
                      if (at < kList) h->all[at] = entry_of(y.x[e], id);
                    }
                  }
              }
          }
        }
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(~0u, sum, d);
        if (lane == 0) h->sum[warp] = sum;
        __syncthreads();
        sum = 0;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) sum += h->sum[w];
        list_mass = static_cast<float>(sum) * 0x1p-40f;
        listed = h->groups <= kList ? h->count : INT32_MAX;
        more = listed > kList ||
               (use_k ? top_k > listed : use_p && listed < a.V && list_mass < top_p * row_mass);
        if (!more) {
          // -- the cuts and the draw on the ranked list
          R.rank_list(listed);
          if (warp == 0) {
            float kept = row_mass, total = 0.0f;
            int keep = use_k ? top_k : listed;
            if (use_k) R.reach(keep, kInf, &kept);
            total = kept;
            if (use_p) keep = R.reach(keep, top_p * kept, &total);
            // below the bar of min-p, or of no weight (masked, or 2^y underflowed): the
            // sums' rounding may leave the target at their mass, and draw none of them
            if (min_p > 0.0f || !(h->w[keep - 1] > 0.0f)) {
              int c = 0;
              for (int i = lane; i < keep; i += 32) c += h->w[i] > 0.0f && h->w[i] >= min_p ? 1 : 0;
              keep = __reduce_add_sync(~0u, c);
              if (min_p > 0.0f) R.reach(keep, kInf, &total);
            }
            if (lane == 0) h->cut = keep, h->total = total, h->pick = INT32_MAX;
          }
          __syncthreads();
          const int keep = h->cut;
          const float total = h->total, target = u * total;
          for (int i = tid; i < keep; i += kThreads) {
            const int id = h->id[i];
            // the mass up to the token, from the lightest, in runs of 32: one by one from
            // the heaviest, equal small weights would all round the same way (500 of
            // 2e-7: off by 2e-6)
            float c = 0.0f;
            bool later = false;
            for (int end = keep; end > 0; end -= 32) {
              const int begin = max(0, end - 32);
              float run = 0.0f;
#pragma unroll 4
              for (int j = end - 1; j >= begin; --j) {
                const int o = h->id[j];
                const float w = h->w[j];
                run += o <= id ? w : 0.0f;
                later |= o > id;
              }
              c += run;
            }
            if (c > target || !later) atomicMin(&h->pick, id);
          }
          __syncthreads();
          for (int i = tid; i < keep; i += kThreads)
            if (h->id[i] == h->pick) {
              a.out_tokens[row] = h->pick;
              if (a.out_probs != nullptr) a.out_probs[row] = h->w[i] / total;
            }
        }
      }
    }
  }
  if (!filtered) return;  // known to every CTA of the row

  // ---- the verdict, and what the search starts from
  {
    const float4(*s)[2] = R.exchange(
        make_float4(R.best, bar_x, list_mass, row_mass),
        make_float4(__int_as_float(listed), __int_as_float(more ? 1 : 0), 0, 0));
    R.best = s[0][0].x, bar_x = s[0][0].y, list_mass = s[0][0].z, row_mass = s[0][0].w;
    listed = __float_as_int(s[0][1].x);
    if (__float_as_int(s[0][1].y) == 0) return;
  }
  Cut cut{-kInf, INT32_MAX, 0.0f};
  constexpr uint32_t kLow = ES == 2 ? 0x7fu : 0x7fffffu;  // key of -inf
  const uint32_t above = key_of<ES>(R.best) + 1;
  // the list's bar bounds the cut where all its tokens were counted
  const uint32_t bar_key = bar_x > -kInf && listed != INT32_MAX ? key_of<ES>(bar_x) : 0;
  const bool counted = listed != INT32_MAX && bar_x > -kInf;  // the bar's list bounds the cut
  const Cut all{-kInf, INT32_MAX, 0.0f};
  if (use_k || use_p) {
    const float need = use_k ? -1.0f : top_p * row_mass;
    const bool below = counted && (use_k ? listed < top_k : list_mass < need);
    const float m_top = below ? list_mass : 0.0f;
    const int c_top = below ? listed : 0;
    // what lies below the floor has less mass than the cut leaves, or top_k
    // tokens are above it: the bar's, where it is that of the top_k-th seed
    float floor_x = -kInf;
    if (!use_k)
      floor_x = R.best + __log2f(0.99f * (1.0f - top_p) * row_mass / a.V) / R.sc;
    else if (top_k <= min(groups, kThreads))
      floor_x = bar_x;
    cut = cut_by_bins<ES>(R, top_k, need, all, below ? bar_x : kInf, m_top, c_top, floor_x);
    R.parity = cut.parity;
    if (!cut.ok) {
      cut = search<ES>(R, top_k, need, kLow, -1, row_mass, a.V, below ? bar_key : above, m_top, c_top,
                       cut.lo, cut.hi);
      R.parity = cut.parity;
    }
  }
  if (use_k && use_p) {
    const Cut k = cut;
    const float need = top_p * k.mass;
    cut = cut_by_bins<ES>(R, 0, need, k, kInf, 0.0f, 0, -kInf);
    R.parity = cut.parity;
    if (!cut.ok) {
      cut = search<ES>(R, 0, need, key_of<ES>(k.t), k.id, k.mass, INT32_MAX, above, 0.0f, 0,
                       cut.lo, cut.hi);
      R.parity = cut.parity;
    }
  }

  // ---- the groups' kept masses, and the draw
  const uint32_t mass0 = peer_addr(&R.stat[0].y, 0);
  auto kept = [&](int i, const uint4& raw) {
    const Vec<ES> x(raw);
    float s = 0;
#pragma unroll
    for (int e = 0; e < N; ++e) {
      const float v = x.x[e], w = R.weight(v);
      const bool on = (w >= min_p) & ((v > cut.t) | ((v == cut.t) & (R.token(i, e) <= cut.id)));
      s += on ? w : 0.0f;
    }
    return s;
  };
  for (int i0 = R.start(); i0 < R.v1; i0 += kThreads * Row<ES>::kLoads) {
    uint4 x[Row<ES>::kLoads];
    float s[Row<ES>::kLoads];
    R.fetch(i0, x);
#pragma unroll
    for (int k = 0; k < Row<ES>::kLoads; ++k) s[k] = kept(i0 + k * kThreads + lane, x[k]);
    auto put = [&](int i, float v) {
      if (i < R.v1)
        asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(mass0 + (i >> a.shift) * 8), "f"(v)
                     : "memory");
    };
    if (G == 8) {
      const float v = fold(s, [](float x, float y) { return x + y; });
      if ((lane & 4) == 0) put(i0 + folded(lane) * kThreads + (lane & 24), v);
    } else {
#pragma unroll
      for (int k = 0; k < Row<ES>::kLoads; ++k) {
        for (int d = 1; d < G; d <<= 1) s[k] += __shfl_xor_sync(~0u, s[k], d);
        if ((lane & (G - 1)) == 0) put(i0 + k * kThreads + lane, s[k]);
      }
    }
  }
  cluster_sync();
  if (rank == 0) draw<ES>(R, a, row, groups, u, cut, min_p);
}

}  // namespace
}  // namespace serve
}  // namespace sv

extern "C" int spec_verify_sample(const void* logits, int64_t row_stride, int32_t N, int32_t V,
                                  int32_t dtype, const float* temperature, const int32_t* top_k,
                                  const float* top_p, const float* min_p, const float* uniforms,
                                  int32_t* out_tokens, float* out_probs, int32_t* dev_error,
                                  void* stream) {
  using namespace sv::serve;
  if (dtype != SV_BF16 && dtype != SV_FP32) return SV_ERR_DTYPE;
  const int es = dtype == SV_BF16 ? 2 : 4;
  if (N < 0 || V < 1 || row_stride < V) return SV_ERR_ARG;
  if (N == 0) return SV_OK;
  if (logits == nullptr || uniforms == nullptr || out_tokens == nullptr ||
      !aligned_to(logits, es) || !aligned_to(uniforms, 4) || !aligned_to(out_tokens, 4) ||
      !null_or_aligned(temperature, 4) || !null_or_aligned(top_k, 4) ||
      !null_or_aligned(top_p, 4) || !null_or_aligned(min_p, 4) || !null_or_aligned(out_probs, 4) ||
      !null_or_aligned(dev_error, 4))
    return SV_ERR_ARG;
  const int64_t row = static_cast<int64_t>(V) * es;
  if (row > SV_SAMPLE_MAX_ROW_BYTES) return SV_ERR_UNSUPPORTED;
  Device d;
  const int rc = device(&d);
  if (rc != SV_OK) return rc;
  const int per = 16 / es, vecs = (V + per - 1) / per + 1;  // one more where the row starts between
  // CTAs a row, each of at least 512 vectors: one an SM for up to a quarter as
  // many rows as SMs (the kernel then has 128 registers a thread; 32 rows under
  // top-p 0.8 48 us, two an SM 52 us), else as many as fit at two an SM (96 rows under top-k 20:
  // three CTAs a row 12 us, four 20 us).
  const bool wide = 4 * static_cast<int64_t>(N) <= d.sms;
  const int C = std::max(1, std::min({kMaxCluster, (wide ? 1 : 2) * d.sms / N, vecs / 512}));
  if (static_cast<int64_t>(N) * C > INT32_MAX) return SV_ERR_UNSUPPORTED;
  const int slice = ((vecs + C - 1) / C + 31) / 32 * 32;
  // groups of 8 vectors; more where that makes over 4096 of them, fewer where a
  // row has fewer than 512
  int shift = 3;
  while (shift < 5 && vecs > 4096 << shift) ++shift;
  while (shift > 0 && vecs < 512 << shift) --shift;
  const int stats = (vecs >> shift) + 2;  // most groups
  const SampleArgs a{static_cast<const char*>(logits), row_stride * es, V, C, slice, shift,
                     temperature, top_k, top_p, min_p, uniforms, out_tokens, out_probs, dev_error};
  const int smem = kHeaderBytes + stats * 8;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (wide)
    return es == 2 ? launch(sample_kernel<2, 1>, dim3(N * C), kThreads, smem, C, false, st, a)
                   : launch(sample_kernel<4, 1>, dim3(N * C), kThreads, smem, C, false, st, a);
  return es == 2 ? launch(sample_kernel<2, 2>, dim3(N * C), kThreads, smem, C, false, st, a)
                 : launch(sample_kernel<4, 2>, dim3(N * C), kThreads, smem, C, false, st, a);
}
