// sv_sample.cu -- one token per row with per-row temperature, top-k, top-p and
// min-p from given random numbers (include/spec_verify_serve.h).
//
// A cluster of C CTAs owns a row: each copies its slice of the row to shared
// memory once (cp.async.bulk, one copy and one barrier a warp), and every pass
// reads it there, so a logit crosses HBM once whatever the filters need.  A
// pass ends with an exchange: each CTA stores its partial into every CTA's
// shared memory, and after the cluster barrier all sum the C partials in rank
// order, so all decide alike.
//
// The kept set is a prefix of the order (value desc, id asc), so its last
// token (value t, id) describes it; min-p is a bar on the weight itself.
//  - Max pass: the row's maximum, and from every warp the largest of its lanes'
//    maxima, 256 seeds a row: R elements are at or above the R-th largest seed.
//  - Collect pass: the tokens at or above that bar go to a list (R = top_k, or
//    192 for top-p alone, whose pass also sums the row's mass).  If the list
//    holds the top-k set, or top_p of the mass, rank 0 finishes on it: ranks by
//    counting, the cuts, the draw.  This is the path of usual rows.
//  - Otherwise a search narrows an interval of values around the cut, three
//    pivots a pass, placed by interpolation, until the interval holds at most
//    kList tokens, which are collected and ranked, or one value (ties).
//    Then one pass draws over the slices.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "sv_host.cuh"
#include "sv_ptx.cuh"

namespace sv {
namespace serve {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;
constexpr float kInf = __builtin_huge_valf();

struct SampleArgs {
  const char* logits;
  int64_t row_bytes;
  int32_t V, C, L;  // CTAs a row, elements a slice
  const float* temperature;
  const int32_t* top_k;
  const float *top_p, *min_p, *uniforms;
  int32_t* out_tokens;
  float* out_probs;
  int32_t* dev_error;
};

constexpr int kSeeds = 256;  // of a row, over all its warps
constexpr int kList = 512;   // most tokens of a list
constexpr int kTopPSeeds = 192;

struct Header {
  float4 slot[2][kMaxCluster][2];  // exchanged partials, two exchanges in turn
  float4 part[kWarps][2];
  uint64_t bar[kWarps];
  uint64_t all[kList];   // rank 0: every CTA's list; key above complemented id
  uint64_t list[kList];  // this CTA's
  float w[kList];        // rank 0: weights and ids, best first
  int32_t id[kList];
  uint16_t seed[kSeeds];
  int32_t count, pick, cut;
  float kept, total;
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

template <int ES>
struct Row {
  static constexpr int N = 16 / ES;
  Header* h;
  const uint4* data;    // this CTA's slice, 16-byte vectors
  int v_first, v_last;  // this warp's run of them
  int first;            // token id of vector 0's element 0 (may start before the slice)
  int begin, end;       // token ids of the slice
  int C, rank, parity = 0;
  float best, sc;       // the row's maximum, log2(e) / T

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

  // The warps' partials (floats a.xyz, integers b.xyz) summed over the CTA in
  // warp order, then over the row in rank order.
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
    for (int i = v_first + (threadIdx.x & 31); i < v_last; i += 32) {
      const Vec<ES> x(data[i]);
#pragma unroll
      for (int e = 0; e < N; ++e)
        if (x.x[e] >= low) {
          const float w = weight(x.x[e]);
#pragma unroll
          for (int j = 0; j < 3; ++j)
            if (x.x[e] >= t[j]) v.m[j] += w, ++v.c[j];
        }
    }
    return total(v);
  }

  __device__ __forceinline__ void append(float x, int id) {
    if (id < begin || id >= end) return;  // what the edge vectors hold beside the slice
    const int at = atomicAdd(&h->count, 1);
    if (at < kList) h->list[at] = entry_of(x, id);
  }

  // This CTA's list (of h->count tokens) into rank 0's, behind those of the
  // ranks before it (`before` tokens).
  __device__ __forceinline__ void send(int before) {
    const int n = h->count;
    uint32_t peer;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(peer) : "r"(smem_addr(h->all)), "r"(0));
    for (int i = threadIdx.x; i < n; i += kThreads)
      asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(peer + (before + i) * 8), "l"(h->list[i])
                   : "memory");
    cluster_sync();
  }

  // Rank 0: weights and ids of the n listed tokens, best first.
  __device__ __forceinline__ void rank_list(int n) {
    for (int i = threadIdx.x; i < n; i += kThreads) {
      const uint64_t e = h->all[i];
      int r = 0;
      for (int j = 0; j < n; ++j) r += h->all[j] > e ? 1 : 0;
      h->w[r] = weight(value_of(e));
      h->id[r] = id_of(e);
    }
    __syncthreads();
  }

  // Warp 0 of rank 0, over the ranked list: the first index (from 1) whose
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
};

// The cut at the k-th best token (need < 0), or where the mass reaches `need`,
// within the tokens at or above key `lo` (of which ties at its value only up
// to id `lo_id`); f_lo >= target > 0 there.  above: a value with fewer than k
// tokens, or less mass than need, at or above it, their count and mass.
template <int ES>
__device__ __noinline__ Cut search(Row<ES>& R, int k, float need, uint32_t lo, int lo_id, float m_lo, int c_lo,
                      uint32_t hi, float m_hi, int c_hi) {
  const bool by_mass = need >= 0.0f;
  constexpr uint32_t kLow = ES == 2 ? 0x7fu : 0x7fffffu;  // key of -inf
  for (int iter = 0; hi - lo > 1 && c_lo - c_hi > kList; ++iter) {
    const float xh = fminf(float_of<ES>(hi), R.best), xl = float_of<ES>(lo);
    uint32_t p[3];
    if (iter < 8 && lo == kLow) {  // no lower end yet: steps of some binades of weight
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
  if (c_lo - c_hi <= kList) {  // the few tokens of the interval, ranked
    __syncthreads();
    if (tid == 0) h->count = 0;
    __syncthreads();
    for (int i = R.v_first + lane; i < R.v_last; i += 32) {
      const Vec<ES> v(R.data[i]);
#pragma unroll
      for (int e = 0; e < N; ++e)
        if (v.x[e] >= tl && (top || v.x[e] < th)) R.append(v.x[e], R.first + i * N + e);
    }
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
    int c = 0;
    for (int i = R.v_first + lane; i < R.v_last; i += 32) {
      const Vec<ES> v(R.data[i]);
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
      for (int i0 = R.v_first; i0 < R.v_last; i0 += 32) {
        const int i = i0 + lane;
        int n = 0;
        if (i < R.v_last) {
          const Vec<ES> v(R.data[i]);
#pragma unroll
          for (int e = 0; e < N; ++e) n += v.x[e] == cut.t ? 1 : 0;
        }
        int inc = n;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
          const int o = __shfl_up_sync(~0u, inc, d);
          if (lane >= d) inc += o;
        }
        if (i < R.v_last && inc - n < left && inc >= left) {
          const Vec<ES> v(R.data[i]);
          int seen = inc - n;
#pragma unroll
          for (int e = 0; e < N; ++e)
            if (v.x[e] == cut.t && ++seen == left) h->pick = R.first + i * N + e;
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
  return cut;
}

template <int ES>
__global__ __launch_bounds__(kThreads) void sample_kernel(const SampleArgs a) {
  extern __shared__ __align__(128) char smem[];
  constexpr int N = 16 / ES;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int row = blockIdx.x / a.C, rank = a.C > 1 ? static_cast<int>(cluster_rank()) : 0;
  Header* h = reinterpret_cast<Header*>(smem);
  char* data = smem + kHeaderBytes;
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");

  // ---- this CTA's slice into shared memory, at the same offset from a
  // 16-byte boundary as in global memory; what the first and last vector hold
  // beside it is -inf, a masked token.  Every warp copies its own run.
  const int64_t e0 = static_cast<int64_t>(rank) * a.L;
  const int n = static_cast<int>(max(static_cast<int64_t>(0),
                                     min(static_cast<int64_t>(a.L), a.V - e0)));
  const char* src = a.logits + row * a.row_bytes + e0 * ES;
  const int lead = static_cast<int>(reinterpret_cast<uintptr_t>(src) & 15);
  const int bytes = lead + n * ES;
  const int nvec = n > 0 ? (bytes + 15) / 16 : 0;
  Row<ES> R;
  R.h = h, R.data = reinterpret_cast<const uint4*>(data);
  const int run = (nvec + kWarps - 1) / kWarps;
  R.v_first = min(nvec, warp * run), R.v_last = min(nvec, R.v_first + run);
  R.first = static_cast<int>(e0) - lead / ES;
  R.begin = static_cast<int>(e0), R.end = static_cast<int>(e0) + n;
  R.C = a.C, R.rank = rank;
  const uint32_t bar = smem_addr(&h->bar[warp]);
  const int b0 = max(R.v_first * 16, lead > 0 ? 16 : 0), b1 = min(R.v_last * 16, bytes / 16 * 16);
  bool timed_out = false;
  if (lane == 0 && b1 > b0) {
    mbar_init(bar, 1);
    fence_mbar_init();
    mbar_arrive_expect_tx(bar, static_cast<uint32_t>(b1 - b0));
    bulk_g2s(smem_addr(data + b0), src - lead + b0, static_cast<uint32_t>(b1 - b0), bar);
  }
  if (R.v_last > R.v_first && lane < 2 * N) {
    const int vec = lane < N ? 0 : nvec - 1;  // the first vector, and the last
    const bool whole = lane < N ? lead == 0 : bytes % 16 == 0 || (vec == 0 && lead > 0);
    if (!whole && vec >= R.v_first && vec < R.v_last) {
      const int at = vec * 16 + (lane % N) * ES;
      const bool in = at >= lead && at < bytes;
      if constexpr (ES == 2)
        *reinterpret_cast<uint16_t*>(data + at) =
            in ? *reinterpret_cast<const uint16_t*>(src - lead + at) : 0xff80u;
      else
        *reinterpret_cast<float*>(data + at) =
            in ? *reinterpret_cast<const float*>(src - lead + at) : -kInf;
    }
  }

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
  if (tid == 0) h->count = 0;
  __syncwarp();
  if (b1 > b0) mbar_wait(bar, 0, timed_out);
  __syncwarp();

  // ---- maximum (NaN wins) and seeds
  float mx = -kInf;
  if constexpr (ES == 2) {
    uint32_t m = 0xff80ff80u;
#pragma unroll 4
    for (int i = R.v_first + lane; i < R.v_last; i += 32) {
      const uint4 v = R.data[i];
      m = bf16x2_max_nan(bf16x2_max_nan(m, bf16x2_max_nan(v.x, v.y)), bf16x2_max_nan(v.z, v.w));
    }
    mx = fmax_nan(bf16lo(m), bf16hi(m));
  } else {
#pragma unroll 4
    for (int i = R.v_first + lane; i < R.v_last; i += 32) {
      const Vec<ES> v(R.data[i]);
      mx = fmax_nan(mx, fmax_nan(fmax_nan(v.x[0], v.x[1]), fmax_nan(v.x[2], v.x[3])));
    }
  }
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");  // every CTA of the row runs
  {
    // the warp's largest lane maxima (upper 16 bits of their keys: a bar may be
    // lower than the seed, never higher), 256 / (8 C) of them, to every CTA
    uint32_t key = key_of<4>(mx) >> 16 << 16 | lane;
    const int per = kSeeds / kWarps / a.C;
    uint32_t mine = 0;
    for (int j = 0; j < per; ++j) {
      const uint32_t top = __reduce_max_sync(~0u, key);
      if (lane == j) mine = top;
      if (key == top) key = 0;
    }
    for (int r = 0; r < a.C && lane < per; ++r) {
      uint32_t peer;
      asm volatile("mapa.shared::cluster.u32 %0, %1, %2;"
                   : "=r"(peer)
                   : "r"(smem_addr(&h->seed[(rank * kWarps + warp) * per + lane])), "r"(r));
      asm volatile("st.shared::cluster.u16 [%0], %1;" ::"r"(peer),
                   "h"(static_cast<uint16_t>(mine >> 16))
                   : "memory");
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) mx = fmax_nan(mx, __shfl_xor_sync(~0u, mx, d));
    if (lane == 0) h->part[warp][0] = make_float4(mx, timed_out ? 1.0f : 0.0f, 0, 0);
    __syncthreads();
    float late = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) mx = fmax_nan(mx, h->part[w][0].x), late += h->part[w][0].y;
    const float4(*s)[2] = R.exchange(make_float4(mx, late, 0, 0), make_float4(0, 0, 0, 0));
    for (int r = 0; r < a.C; ++r) {
      mx = fmax_nan(mx, s[r][0].x);
      if (s[r][0].y != 0.0f) err |= SV_DEVERR_TIMEOUT;
    }
  }
  if (!(mx > -kInf && mx < kInf)) err |= SV_DEVERR_NAN;
  if (err != 0) {  // the same in every CTA of the row
    if (rank == 0 && tid == 0) {
      a.out_tokens[row] = -1;
      if (a.out_probs != nullptr) a.out_probs[row] = 0.0f;
      if (a.dev_error != nullptr) atomicOr(a.dev_error, static_cast<int32_t>(err));
    }
    return;
  }
  R.best = mx;

  Cut cut{-kInf, INT32_MAX, 0.0f};
  const bool use_k = top_k > 0, use_p = top_p < 1.0f;
  if (use_k || use_p || min_p > 0.0f) {
    // ---- the bar and the tokens at or above it
    float bar_x;
    if (!use_k && !use_p) {  // min-p alone: its own bar, a little lower
      const float y = __log2f(min_p) - 0.001f;
      bar_x = fmaf(y, 1.0f / R.sc, mx) - fabsf(mx) * 1e-6f;
    } else {  // the R-th largest seed, by bisection over their 16 bits
      const int want = use_k ? min(top_k, kSeeds) : kTopPSeeds;
      uint32_t s[kSeeds / 32];
#pragma unroll
      for (int j = 0; j < kSeeds / 32; ++j) s[j] = h->seed[j * 32 + lane];
      uint32_t at = 0;
      for (uint32_t bit = 0x8000u; bit != 0; bit >>= 1) {
        int c = 0;
#pragma unroll
        for (int j = 0; j < kSeeds / 32; ++j) c += s[j] >= (at | bit) ? 1 : 0;
        if (__reduce_add_sync(~0u, c) >= want) at |= bit;
      }
      bar_x = at <= 0x7fu ? -kInf : float_of<4>(at << 16);
    }
    const bool need_z = !use_k && use_p;
    typename Row<ES>::Sums v{{0, 0, 0}, {0, 0, 0}};
    for (int i = R.v_first + lane; i < R.v_last; i += 32) {
      const uint4 raw = R.data[i];
      if (need_z) {
        const Vec<ES> x(raw);
#pragma unroll
        for (int e = 0; e < N; ++e) {
          const float w = R.weight(x.x[e]);
          v.m[0] += w;
          if (x.x[e] >= bar_x) v.m[1] += w, R.append(x.x[e], R.first + i * N + e);
        }
      } else {
        float top;
        if constexpr (ES == 2) {
          const uint32_t m = bf16x2_max_nan(bf16x2_max_nan(raw.x, raw.y), bf16x2_max_nan(raw.z, raw.w));
          top = fmaxf(bf16lo(m), bf16hi(m));
        } else {
          const Vec<ES> x(raw);
          top = fmaxf(fmaxf(x.x[0], x.x[1]), fmaxf(x.x[2], x.x[3]));
        }
        if (top >= bar_x) {
          const Vec<ES> x(raw);
#pragma unroll
          for (int e = 0; e < N; ++e)
            if (x.x[e] >= bar_x) v.m[1] += R.weight(x.x[e]), R.append(x.x[e], R.first + i * N + e);
        }
      }
    }
    __syncthreads();
    // every CTA's count (at .w) beside the masses
    v.c[0] = tid == 0 ? h->count : 0;
    const int parity = R.parity;
    const typename Row<ES>::Sums s = R.total(v);
    const int listed = s.c[0];
    const bool enough = listed <= kList && (use_k ? top_k <= listed : !use_p || s.m[1] >= top_p * s.m[0]);
    if (enough) {
      // ---- rank 0 finishes on the list
      int before = 0;
      for (int r = 0; r < rank; ++r) before += __float_as_int(h->slot[parity][r][1].x);
      R.send(before);
      if (rank != 0) return;
      R.rank_list(listed);
      if (warp == 0) {
        float kept, total;
        int keep = use_k ? top_k : listed;
        R.reach(keep, kInf, &kept);
        if (!use_k) kept = s.m[0];
        if (use_p) keep = R.reach(keep, top_p * kept, &total);
        if (min_p > 0.0f) {
          int c = 0;
          for (int i = lane; i < keep; i += 32) c += h->w[i] >= min_p ? 1 : 0;
          keep = __reduce_add_sync(~0u, c);
        }
        R.reach(keep, kInf, &total);
        if (lane == 0) h->cut = keep, h->total = total, h->pick = INT32_MAX;
      }
      __syncthreads();
      const int keep = h->cut;
      const float total = h->total, target = u * total;
      for (int i = tid; i < keep; i += kThreads) {
        const int id = h->id[i];
        float c = h->w[i];
        bool later = false;
        for (int j = 0; j < keep; ++j) {
          if (h->id[j] < id) c += h->w[j];
          later |= h->id[j] > id;
        }
        if (c > target || !later) atomicMin(&h->pick, id);
      }
      __syncthreads();
      for (int i = tid; i < keep; i += kThreads)
        if (h->id[i] == h->pick) {
          a.out_tokens[row] = h->pick;
          if (a.out_probs != nullptr) a.out_probs[row] = h->w[i] / total;
        }
      return;
    }
    // ---- the cuts by search, from the bar on the side of it that they lie on
    constexpr uint32_t kLow = ES == 2 ? 0x7fu : 0x7fffffu;  // key of -inf
    const uint32_t bar_key = bar_x > -kInf ? key_of<ES>(bar_x) : 0, above = key_of<ES>(mx) + 1;
    if (use_k) {
      if (listed >= top_k && bar_key != 0)
        cut = search<ES>(R, top_k, -1.0f, bar_key, -1, 0.0f, listed, above, 0.0f, 0);
      else if (bar_key != 0)
        cut = search<ES>(R, top_k, -1.0f, kLow, -1, 0.0f, a.V, bar_key, s.m[1], listed);
      else
        cut = search<ES>(R, top_k, -1.0f, kLow, -1, 0.0f, a.V, above, 0.0f, 0);
      if (use_p)
        cut = search<ES>(R, 0, top_p * cut.mass, key_of<ES>(cut.t), cut.id, cut.mass, INT32_MAX,
                         above, 0.0f, 0);
    } else if (use_p) {
      const float need = top_p * s.m[0];
      if (bar_key == 0)
        cut = search<ES>(R, 0, need, kLow, -1, s.m[0], a.V, above, 0.0f, 0);
      else if (s.m[1] >= need)
        cut = search<ES>(R, 0, need, bar_key, -1, s.m[1], listed, above, 0.0f, 0);
      else
        cut = search<ES>(R, 0, need, kLow, -1, s.m[0], a.V, bar_key, s.m[1], listed);
    }
  }

  // ---- the draw: masses of the warps' runs, the run that holds u * total,
  // and a walk along it
  auto weight = [&](float x, int id) {
    if (!(x > cut.t || (x == cut.t && id <= cut.id))) return 0.0f;
    const float w = R.weight(x);
    return w >= min_p ? w : 0.0f;
  };
  float m = 0;
  for (int i = R.v_first + lane; i < R.v_last; i += 32) {
    const Vec<ES> v(R.data[i]);
#pragma unroll
    for (int e = 0; e < N; ++e) m += weight(v.x[e], R.first + i * N + e);
  }
  m = warp_sum(m);
  __syncthreads();
  if (lane == 0) h->part[warp][0].x = m;
  __syncthreads();
  float cta = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) cta += h->part[w][0].x;
  const float4(*s)[2] = R.exchange(make_float4(cta, 0, 0, 0), make_float4(0, 0, 0, 0));
  float total = 0;
  for (int r = 0; r < a.C; ++r) total += s[r][0].x;
  const float target = u * total;
  int owner = -1;
  float below = 0, run_sum = 0;
  for (int r = 0; r < a.C; ++r) {
    const float x = s[r][0].x;
    if (x > 0.0f) owner = r, below = run_sum;
    run_sum += x;
    if (x > 0.0f && run_sum > target) break;
  }
  if (rank != owner) return;
  int own_warp = -1;
  float at = below, base = below;
  for (int w = 0; w < kWarps; ++w) {
    const float x = h->part[w][0].x;
    if (x > 0.0f) own_warp = w, base = at;
    at += x;
    if (x > 0.0f && at > target) break;
  }
  if (warp != own_warp) return;
  int found = -1, last = -1;
  float fw = 0, lw = 0, cum = base;
  for (int i0 = R.v_first; i0 < R.v_last && found < 0; i0 += 32) {
    const int i = i0 + lane;
    float w[N], k = 0;
#pragma unroll
    for (int e = 0; e < N; ++e) w[e] = 0;
    if (i < R.v_last) {
      const Vec<ES> v(R.data[i]);
#pragma unroll
      for (int e = 0; e < N; ++e) w[e] = weight(v.x[e], R.first + i * N + e), k += w[e];
    }
    float inc = k;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const float o = __shfl_up_sync(~0u, inc, d);
      if (lane >= d) inc += o;
    }
    float c = cum + (inc - k);
    int mine_id = -1, mine_last = -1;
    float mine_w = 0, mine_lw = 0;
#pragma unroll
    for (int e = 0; e < N; ++e) {
      c += w[e];
      if (w[e] > 0.0f) {
        mine_last = R.first + i * N + e, mine_lw = w[e];
        if (mine_id < 0 && c > target) mine_id = mine_last, mine_w = w[e];
      }
    }
    const unsigned hit = __ballot_sync(~0u, mine_id >= 0);
    const unsigned any = __ballot_sync(~0u, mine_last >= 0);
    if (hit != 0) {
      const int l = __ffs(hit) - 1;
      found = __shfl_sync(~0u, mine_id, l), fw = __shfl_sync(~0u, mine_w, l);
    }
    if (any != 0) {
      const int l = 31 - __clz(any);
      last = __shfl_sync(~0u, mine_last, l), lw = __shfl_sync(~0u, mine_lw, l);
    }
    cum += __shfl_sync(~0u, inc, 31);
  }
  if (found < 0) found = last, fw = lw;  // the sums' rounding left the target past the run
  if (lane == 0) {
    a.out_tokens[row] = found;
    if (a.out_probs != nullptr) a.out_probs[row] = fw / total;
  }
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
  // slices of at most 40 KB while eight CTAs suffice: five CTAs fit an SM, so
  // some copy while others compute
  int C = 1;
  while (C < kMaxCluster && row > static_cast<int64_t>(C) * 40960) C *= 2;
  if (static_cast<int64_t>(N) * C > INT32_MAX) return SV_ERR_UNSUPPORTED;
  const int per = 16 / es;
  const int L = ((V + C - 1) / C + per - 1) / per * per;
  const SampleArgs a{static_cast<const char*>(logits), row_stride * es, V, C, L, temperature,
                     top_k, top_p, min_p, uniforms, out_tokens, out_probs, dev_error};
  const int smem = kHeaderBytes + L * es + 32;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return es == 2 ? launch(sample_kernel<2>, dim3(N * C), kThreads, smem, C, false, st, a)
                 : launch(sample_kernel<4>, dim3(N * C), kThreads, smem, C, false, st, a);
}
