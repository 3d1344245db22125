// sv_sample.cu -- one token per row with per-row temperature, top-k, top-p and
// min-p from given random numbers (include/spec_verify_serve.h).
//
// A cluster of C CTAs owns a row: each copies its slice of the row to shared
// memory once (cp.async.bulk), and every later pass reads it there, so a logit
// crosses HBM once whatever the filters need.  A pass ends with an exchange:
// each CTA stores its partial into every CTA's shared memory, and after the
// cluster barrier all sum the C partials in rank order, so all decide alike.
//
// The kept set is a prefix of the order (value desc, id asc): a value t, and
// how many of the tokens that equal t stay (the lowest ids).  t is found by
// bisection over the order-preserving bits of a float (16 steps for bf16, 32
// for fp32): for top-k on the count of x >= t, for top-p on their mass.  min-p
// is a bar on the weight itself.
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

struct Header {
  float4 slot[2][kMaxCluster];  // exchanged partials, two exchanges in turn
  float4 part[kWarps];
  uint64_t bar;
  int32_t id;
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
__device__ __forceinline__ int warp_sum(int v) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(~0u, v, d);
  return v;
}

template <int ES>
struct Row {
  static constexpr int N = 16 / ES;
  Header* h;
  const uint4* data;  // this CTA's slice, 16-byte vectors
  int nvec, v_first, v_last;  // its vectors, and this warp's run of them
  int first;                  // token id of vector 0's element 0 (may start before the slice)
  int C, rank, parity = 0;

  // Every CTA's partial, in rank order, to every thread.
  __device__ __forceinline__ const float4* exchange(float4 mine) {
    Header* hh = h;
    if (threadIdx.x < C)
      store_peer(smem_addr(&hh->slot[parity][rank]), threadIdx.x, mine);
    cluster_sync();
    const float4* s = hh->slot[parity];
    parity ^= 1;
    return s;
  }

  // A warp's partial of each pass (x: sum of floats, y: of ints' bits) summed
  // over the CTA in warp order; every thread gets the sum.
  __device__ __forceinline__ float4 cta_sum(float mass, int count) {
    __syncthreads();
    if ((threadIdx.x & 31) == 0)
      h->part[threadIdx.x >> 5] = make_float4(mass, __int_as_float(count), 0, 0);
    __syncthreads();
    float m = 0;
    int c = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) m += h->part[w].x, c += __float_as_int(h->part[w].y);
    return make_float4(m, __int_as_float(c), 0, 0);
  }

  __device__ __forceinline__ void total(float mass, int count, float* all_mass, int* all_count) {
    const float4* s = exchange(cta_sum(warp_sum(mass), warp_sum(count)));
    float m = 0;
    int c = 0;
    for (int r = 0; r < C; ++r) m += s[r].x, c += __float_as_int(s[r].y);
    *all_mass = m, *all_count = c;
  }

  // Mass and count of the tokens with x >= t.
  __device__ __forceinline__ void at_least(float t, float best, float sc, float* mass, int* count) {
    float m = 0;
    int c = 0;
    for (int i = v_first + (threadIdx.x & 31); i < v_last; i += 32) {
      const Vec<ES> v(data[i]);
#pragma unroll
      for (int e = 0; e < N; ++e)
        if (v.x[e] >= t) m += weight_of(v.x[e], best, sc), ++c;
    }
    total(m, c, mass, count);
  }
};

template <int ES>
__global__ __launch_bounds__(kThreads) void sample_kernel(const SampleArgs a) {
  extern __shared__ __align__(128) char smem[];
  constexpr int N = 16 / ES;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int row = blockIdx.x / a.C, rank = a.C > 1 ? static_cast<int>(cluster_rank()) : 0;
  Header* h = reinterpret_cast<Header*>(smem);
  char* data = smem + kHeaderBytes;

  // ---- this CTA's slice into shared memory, at the same offset from a
  // 16-byte boundary as in global memory; what the first and last vector hold
  // beside it is -inf, a masked token.
  const int64_t e0 = static_cast<int64_t>(rank) * a.L;
  const int n = static_cast<int>(max(static_cast<int64_t>(0),
                                     min(static_cast<int64_t>(a.L), a.V - e0)));
  const char* src = a.logits + row * a.row_bytes + e0 * ES;
  const int lead = static_cast<int>(reinterpret_cast<uintptr_t>(src) & 15);
  const int bytes = lead + n * ES;
  const int nvec = n > 0 ? (bytes + 15) / 16 : 0;
  const int b0 = lead > 0 ? 16 : 0, b1 = bytes / 16 * 16;  // whole vectors: bytes [b0, b1)
  const uint32_t bar = smem_addr(&h->bar);
  bool timed_out = false;
  if (tid == 0) {
    mbar_init(bar, 1);
    fence_mbar_init();
    if (b1 > b0) {
      mbar_arrive_expect_tx(bar, static_cast<uint32_t>(b1 - b0));
      bulk_g2s(smem_addr(data + b0), src - lead + b0, static_cast<uint32_t>(b1 - b0), bar);
    }
  }
  for (int i = tid; i < 2 * N; i += kThreads) {
    const int vec = i < N ? 0 : nvec - 1;  // the first vector, and the last
    if (vec < 0 || (i < N ? b0 == 0 : b1 == nvec * 16) || (i >= N && vec == 0 && b0 > 0)) continue;
    const int at = vec * 16 + (i % N) * ES;
    const bool in = at >= lead && at < bytes;
    if constexpr (ES == 2)
      *reinterpret_cast<uint16_t*>(data + at) =
          in ? *reinterpret_cast<const uint16_t*>(src - lead + at) : 0xff80u;
    else
      *reinterpret_cast<float*>(data + at) =
          in ? *reinterpret_cast<const float*>(src - lead + at) : -kInf;
  }
  __syncthreads();
  cluster_sync();  // every CTA of the row runs: its shared memory can be written
  if (b1 > b0) mbar_wait(bar, 0, timed_out);

  Row<ES> R;
  R.h = h, R.data = reinterpret_cast<const uint4*>(data), R.nvec = nvec;
  const int run = (nvec + kWarps - 1) / kWarps;
  R.v_first = min(nvec, warp * run), R.v_last = min(nvec, R.v_first + run);
  R.first = static_cast<int>(e0) - lead / ES;
  R.C = a.C, R.rank = rank;

  // ---- the row's settings
  const float T = a.temperature != nullptr ? a.temperature[row] : 1.0f;
  const int top_k = a.top_k != nullptr ? a.top_k[row] : 0;
  const float top_p = a.top_p != nullptr ? a.top_p[row] : 1.0f;
  const float min_p = a.min_p != nullptr ? a.min_p[row] : 0.0f;
  const float u = a.uniforms[row];
  uint32_t err = 0;
  if (!(T >= 0.0f && T < kInf) || !(top_p > 0.0f && top_p <= 1.0f) ||
      !(min_p >= 0.0f && min_p <= 1.0f) || !(u >= 0.0f && u < 1.0f))
    err = SV_DEVERR_PARAM;

  // ---- maximum (NaN wins)
  float mx = -kInf;
  for (int i = R.v_first + lane; i < R.v_last; i += 32) {
    const Vec<ES> v(R.data[i]);
#pragma unroll
    for (int e = 0; e < N; ++e) mx = fmax_nan(mx, v.x[e]);
  }
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) mx = fmax_nan(mx, __shfl_xor_sync(~0u, mx, d));
  if (lane == 0) h->part[warp].x = mx;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kWarps; ++w) mx = fmax_nan(mx, h->part[w].x);
  {
    const float4* s = R.exchange(make_float4(mx, timed_out ? 1.0f : 0.0f, 0, 0));
    for (int r = 0; r < a.C; ++r) {
      mx = fmax_nan(mx, s[r].x);
      if (s[r].y != 0.0f) err |= SV_DEVERR_TIMEOUT;
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

  // ---- threshold: keep x > t, of x == t the lowest `ties` ids, and of those
  // the ones with weight >= min_p
  const bool greedy = T == 0.0f;
  const float sc = greedy ? 1.0f : fminf(1.4426950408889634f / T, 3.0e38f);
  float t = -kInf;
  int64_t ties = INT32_MAX;
  if (greedy) {
    t = mx, ties = 1;
  } else {
    uint32_t lo = key_of<ES>(-kInf);
    const uint32_t top = key_of<ES>(mx) + 1;
    float kept = 0;  // mass of the top-k set
    if (top_k > 0 && top_k < a.V) {
      uint32_t hi = top;  // count(x >= lo) >= k > count(x >= hi)
      float above = 0;
      int n_above = 0;
      while (hi - lo > 1) {
        const uint32_t mid = lo + (hi - lo) / 2;
        float m;
        int c;
        R.at_least(float_of<ES>(mid), mx, sc, &m, &c);
        if (c >= top_k) lo = mid;
        else hi = mid, above = m, n_above = c;
      }
      t = float_of<ES>(lo), ties = top_k - n_above;
      kept = above + static_cast<float>(ties) * weight_of(t, mx, sc);
    } else if (top_p < 1.0f) {
      int c;
      R.at_least(-kInf, mx, sc, &kept, &c);
    }
    if (top_p < 1.0f) {
      const float need = top_p * kept;
      const uint32_t floor_key = lo;
      uint32_t hi = top;  // mass(x >= lo) >= need > mass(x >= hi)
      float above = 0;
      while (hi - lo > 1) {
        const uint32_t mid = lo + (hi - lo) / 2;
        float m;
        int c;
        R.at_least(float_of<ES>(mid), mx, sc, &m, &c);
        if (m >= need) lo = mid;
        else hi = mid, above = m;
      }
      t = float_of<ES>(lo);
      const float w = weight_of(t, mx, sc);
      const float more = w > 0.0f ? ceilf((need - above) / w) : 1.0f;
      const int64_t want = static_cast<int64_t>(fminf(fmaxf(more, 1.0f), 2.0e9f));
      ties = lo == floor_key ? min(ties, want) : want;
    }
  }

  // ---- the id of the last tie that stays
  int last_tie = INT32_MAX;
  if (ties < INT32_MAX) {
    int c = 0;
    for (int i = R.v_first + lane; i < R.v_last; i += 32) {
      const Vec<ES> v(R.data[i]);
#pragma unroll
      for (int e = 0; e < N; ++e) c += v.x[e] == t ? 1 : 0;
    }
    const int mine = warp_sum(c);
    const float4* s = R.exchange(R.cta_sum(0.0f, mine));
    int before = 0, all = 0;
    for (int r = 0; r < a.C; ++r) {
      if (r < rank) before += __float_as_int(s[r].y);
      all += __float_as_int(s[r].y);
    }
    for (int w = 0; w < warp; ++w) before += __float_as_int(h->part[w].y);
    if (tid == 0) h->id = -1;
    __syncthreads();
    if (ties < all && before < ties && before + mine >= ties) {  // this warp's run holds it
      int left = static_cast<int>(ties) - before;
      for (int i0 = R.v_first; i0 < R.v_last; i0 += 32) {
        const int i = i0 + lane;
        int k = 0;
        if (i < R.v_last) {
          const Vec<ES> v(R.data[i]);
#pragma unroll
          for (int e = 0; e < N; ++e) k += v.x[e] == t ? 1 : 0;
        }
        int inc = k;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
          const int o = __shfl_up_sync(~0u, inc, d);
          if (lane >= d) inc += o;
        }
        if (i < R.v_last && inc - k < left && inc >= left) {
          const Vec<ES> v(R.data[i]);
          int seen = inc - k;
#pragma unroll
          for (int e = 0; e < N; ++e)
            if (v.x[e] == t && ++seen == left) h->id = R.first + i * N + e;
        }
        const int step = __shfl_sync(~0u, inc, 31);
        if (step >= left) break;
        left -= step;
      }
    }
    __syncthreads();
    const float4* f = R.exchange(make_float4(__int_as_float(h->id), 0, 0, 0));
    if (ties < all)
      for (int r = 0; r < a.C; ++r) last_tie = min(last_tie, __float_as_int(f[r].x) < 0 ? INT32_MAX : __float_as_int(f[r].x));
  }

  // ---- the draw: masses of the warps' runs, the run that holds u * total,
  // and a walk along it
  auto weight = [&](float x, int id) {
    if (!(x > t || (x == t && id <= last_tie))) return 0.0f;
    const float w = weight_of(x, mx, sc);
    return w >= min_p ? w : 0.0f;
  };
  float m = 0;
  for (int i = R.v_first + lane; i < R.v_last; i += 32) {
    const Vec<ES> v(R.data[i]);
#pragma unroll
    for (int e = 0; e < N; ++e) m += weight(v.x[e], R.first + i * N + e);
  }
  const float mine = warp_sum(m);
  const float4* s = R.exchange(R.cta_sum(mine, 0));
  float total = 0;
  for (int r = 0; r < a.C; ++r) total += s[r].x;
  const float target = u * total;
  int owner = -1;
  float below = 0, run_sum = 0;
  for (int r = 0; r < a.C; ++r) {
    if (s[r].x > 0.0f) owner = r, below = run_sum;
    run_sum += s[r].x;
    if (s[r].x > 0.0f && run_sum > target) break;
  }
  if (rank == owner) {
    int own_warp = -1;
    float at = below, base = below;
    for (int w = 0; w < kWarps; ++w) {
      const float x = h->part[w].x;
      if (x > 0.0f) own_warp = w, base = at;
      at += x;
      if (x > 0.0f && at > target) break;
    }
    if (warp == own_warp) {
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
