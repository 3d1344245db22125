// sv_rope.cu -- rotary positions, alone and on the way into a paged cache of 16, 32
// or 8 bits (include/spec_verify_serve.h).
//
// A head's first `rotary` dimensions are pairs turned by position * frequency.  The
// angle is formed in whole numbers: frequencies are turns a position in units of
// 2^-64, so the product modulo 2^64 is the fraction of a turn, exact to 2^-33 of a
// turn at position 2^31, where a product in fp32 is off by whole radians from some
// 10^7 on.  Its top 32 bits go through sincospi, an error of 2^-24 of the angle.
//
// Many rows: a warp a row.  It forms the row's sines once, two a lane, keeps those of its
// eight dimensions in registers, and streams the row's heads, four loads of 512 bytes in
// flight: queries, keys, values, of which only the cached ones pay for their codes.  The
// halves of a pair meet by shuffles, and an 8-bit row's largest magnitude too.  Few rows
// would leave most warps without one: there a group of 8, 16 or 32 lanes holds one vector
// (a head of a row), CTAs hold vectors of one kind and form their rows' sines in shared
// memory while the loads are in flight.  Bound by the bytes, each read and written once:
// 16,384 rows of 32/8 heads of 128 into an 8-bit cache 65 us, 5.7 TB/s, 0.84 of the measured
// copy rate (a group a vector there, its addresses and sines formed anew: 101 to 128 us);
// 512 rows 6.2 us called, of which the launch is most.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <type_traits>

#include "sv_e4m3.cuh"
#include "sv_host.cuh"
#include "sv_ptx.cuh"

namespace sv {
namespace serve {
namespace {

constexpr int kRopeThreads = 256;
constexpr int kRopeFlight = 4;  // loads of a lane in flight

struct RopeArgs {
  const char *q, *k, *v;
  int64_t q_row, q_head, k_row, k_head, v_row, v_head;  // bytes
  char* oq;
  int64_t oq_row, oq_head;  // bytes
  const int32_t* positions;
  const int64_t* freqs;
  const int64_t* slots;
  char *k_cache, *v_cache;
  int64_t block, token, head;  // bytes
  int8_t *k_exps, *v_exps;
  int64_t e_block, e_token, e_head;
  int64_t n_slots;
  int32_t* dev_error;
  int32_t n_rows, heads, kv_heads, dim, half;  // half: pairs
  int32_t q_ctas, kv_ctas;                     // CTAs of queries; of keys, and as many of values
  int32_t page, lanes_log2;
  float amplitude;
  FastDiv by_heads, by_kv_heads, by_half, by_page;
};

// Pairs of a row with those that a spread group of eight may fill.
__host__ __device__ inline int padded_pairs(int half) { return (half + 7) & ~7; }

// Bytes of the sines of the most rows that `vectors` neighbouring vectors lie in.
int rope_smem(int vectors, int per_row, int half) {
  const int rows = (vectors + per_row - 2) / per_row + 1;
  return std::min(rows, vectors) * padded_pairs(half) * static_cast<int>(sizeof(float2));
}

template <typename T>
__device__ __forceinline__ float to_float(T x) { return x; }
template <>
__device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }
template <typename T>
__device__ __forceinline__ T from_float(float x) { return x; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_float(float x) { return __float2bfloat16_rn(x); }

struct Yes { static constexpr bool value = true; };
struct No { static constexpr bool value = false; };

// Eight dimensions as they lie in memory.
template <typename T>
struct Eight {
  static constexpr int kWords = 8 * sizeof(T) / 4;
  uint32_t w[kWords];
  __device__ __forceinline__ void load(const char* p) {
#pragma unroll
    for (int i = 0; i < kWords / 4; ++i) {
      const uint4 x = reinterpret_cast<const uint4*>(p)[i];
      w[i * 4] = x.x, w[i * 4 + 1] = x.y, w[i * 4 + 2] = x.z, w[i * 4 + 3] = x.w;
    }
  }
  __device__ __forceinline__ void store(char* p) const {
#pragma unroll
    for (int i = 0; i < kWords / 4; ++i)
      reinterpret_cast<uint4*>(p)[i] = make_uint4(w[i * 4], w[i * 4 + 1], w[i * 4 + 2], w[i * 4 + 3]);
  }
  __device__ __forceinline__ void get(float* x) const {
    if constexpr (sizeof(T) == 2) {
#pragma unroll
      for (int i = 0; i < 4; ++i) x[2 * i] = bf16lo(w[i]), x[2 * i + 1] = bf16hi(w[i]);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = __uint_as_float(w[i]);
    }
  }
  __device__ __forceinline__ void set(const float* x) {
    if constexpr (sizeof(T) == 2) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[i]) : "f"(x[2 * i + 1]), "f"(x[2 * i]));
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) w[i] = __float_as_uint(x[i]);
    }
  }
};

__device__ __forceinline__ uint64_t two(float lo, float hi) {
  uint64_t v;
  asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(lo), "f"(hi));
  return v;
}
// a * b + c * d of two floats at once
__device__ __forceinline__ void turn2(float* y, const float* a, const float* b, const float* c, const float* d) {
  uint64_t v;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(v) : "l"(two(c[0], c[1])), "l"(two(d[0], d[1])));
  asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(v) : "l"(two(a[0], a[1])), "l"(two(b[0], b[1])));
  asm("mov.b64 {%0, %1}, %2;" : "=f"(y[0]), "=f"(y[1]) : "l"(v));
}

// (cos, sin) of a position and a frequency, times the amplitude.
__device__ __forceinline__ float2 sine_of(int32_t position, int64_t freq, float amplitude) {
  const uint64_t turns = static_cast<uint64_t>(freq) * static_cast<uint64_t>(static_cast<int64_t>(position));
  float s, c;
  sincospif(static_cast<float>(static_cast<int32_t>(turns >> 32)) * 0x1p-31f, &s, &c);
  return make_float2(c * amplitude, s * amplitude);
}
// Where pair i of a row lies among its float2.  A lane reads four units of two pairs in a
// row, so units are spread over the banks: without it eight lanes' reads meet in two of
// the eight places.
__device__ __forceinline__ int sine_place(int i) {
  return (i & ~7) | (((i >> 1 & 3) ^ (i >> 4 & 3)) << 1) | (i & 1);
}
// A lane's eight dimensions from d0: cos, and sin with the sign that its partner takes.
template <bool PAIRS>
__device__ __forceinline__ void lane_sines(const float4* sines, int d0, int half, float* co, float* si) {
#pragma unroll
  for (int e = 0; e < 8; e += PAIRS ? 4 : 2) {  // two pairs
    const int d = d0 + e;
    const float4 z = sines[sine_place(PAIRS ? d >> 1 : d < half ? d : d - half) >> 1];
    if constexpr (PAIRS) {
      co[e] = co[e + 1] = z.x, co[e + 2] = co[e + 3] = z.z;
      si[e] = -z.y, si[e + 1] = z.y, si[e + 2] = -z.w, si[e + 3] = z.w;
    } else {
      const float sign = d < half ? -1.0f : 1.0f;
      co[e] = z.x, si[e] = sign * z.y, co[e + 1] = z.z, si[e + 1] = sign * z.w;
    }
  }
}
// The lanes with the other halves of lane's pairs, of its first and its last four
// dimensions: whole chunks away, or four dimensions more where the pairs are an odd
// number of fours, whose words lie in the other half of their chunks.
struct Partners {
  int first, last;
  bool crossed;
};
__device__ __forceinline__ Partners partners_of(int lane, int c, int half) {
  auto other = [&](int d) { return lane - c + ((d < half ? d + half : d < 2 * half ? d - half : d) >> 3); };
  return {other(c * 8), other(c * 8 + 4), (half & 4) != 0};
}
// Turns a lane's chunk.
template <typename T, bool PAIRS>
__device__ __forceinline__ void turn_chunk(const Eight<T>& raw, const Partners& p, bool turned, const float* co,
                                           const float* si, float* y) {
  float there[8];
  if constexpr (PAIRS) {
#pragma unroll
    for (int e = 0; e < 8; ++e) there[e] = y[e ^ 1];
  } else {
    constexpr int kWords = Eight<T>::kWords;
    Eight<T> w;
#pragma unroll
    for (int i = 0; i < kWords; ++i)
      w.w[i] = __shfl_sync(~0u, p.crossed ? raw.w[i ^ kWords / 2] : raw.w[i], i < kWords / 2 ? p.first : p.last);
    w.get(there);
  }
  if (turned) {
#pragma unroll
    for (int e = 0; e < 8; e += 2) turn2(y + e, y + e, co + e, there + e, si + e);
  }
}
// The exponent of a vector that `lanes` lanes hold eight elements of, `counts`: this
// lane's are of it.  Infinities become NaN, and neither counts.
__device__ __forceinline__ int vector_exponent(float* y, const bool* counts, int lanes) {
  constexpr float kInf = __builtin_huge_valf();
  auto largest = [&]() {
    float top = 0.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (counts[e]) top = fmaxf(top, fabsf(y[e]));
    for (int d = lanes >> 1; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, d));
    return top;
  };
  float top = largest();
  if (__any_sync(~0u, top == kInf)) {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (fabsf(y[e]) == kInf) y[e] = __uint_as_float(0x7fffffffu);
    top = largest();
  }
  return e4m3_exponent(top);
}

// A warp a row; every vector starts on 16 bytes, dimensions and pairs are whole chunks.
template <typename T, bool QUANT, bool PAIRS>
__global__ __launch_bounds__(kRopeThreads, 4) void rope_row_kernel(const __grid_constant__ RopeArgs a) {
  extern __shared__ __align__(16) float4 row_sines[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int row = blockIdx.x * (kRopeThreads / 32) + warp;
  if (row >= a.n_rows) return;  // no barrier but the warp's own below
  const int lanes = 1 << a.lanes_log2, c = lane & (lanes - 1), group = lane >> a.lanes_log2,
            each = 32 >> a.lanes_log2;  // vectors of a load
  const int d0 = c * 8;
  const bool mine = d0 < a.dim, turned = d0 < 2 * a.half;
  const Partners partner = partners_of(lane, c, a.half);
  float4* const sines = row_sines + warp * (padded_pairs(a.half) >> 1);
  float co[8], si[8];
  if (a.half > 0) {
    const int32_t position = __ldg(a.positions + row);
    for (int i = lane; i < a.half; i += 32)
      reinterpret_cast<float2*>(sines)[sine_place(i)] = sine_of(position, __ldg(a.freqs + i), a.amplitude);
    __syncwarp();
    if (turned) lane_sines<PAIRS>(sines, d0, a.half, co, si);
  }
  // heads of one kind, `step` bytes apart, to heads `out_step` bytes apart
  auto heads = [&](auto rotate, auto codes, const char* in, int64_t step, int count, char* out, int64_t out_step,
                   int8_t* exps, int64_t e_step) {
    in += group * step + d0 * sizeof(T), out += group * out_step + d0 * (decltype(codes)::value ? 1 : sizeof(T));
    exps += group * e_step;
    for (int h0 = 0; h0 < count; h0 += kRopeFlight * each) {
      Eight<T> raw[kRopeFlight];
#pragma unroll
      for (int u = 0; u < kRopeFlight; ++u)
        if (h0 + u * each + group < count && mine) raw[u].load(in + u * each * step);
#pragma unroll
      for (int u = 0; u < kRopeFlight; ++u) {
        if (u > 0 && h0 + u * each >= count) break;  // the whole warp
        const bool on = h0 + u * each + group < count && mine;
        float y[8];
        if constexpr (decltype(rotate)::value || decltype(codes)::value) raw[u].get(y);
        if constexpr (decltype(rotate)::value) turn_chunk<T, PAIRS>(raw[u], partner, turned, co, si, y);
        if constexpr (decltype(codes)::value) {
          const bool counts[8] = {on, on, on, on, on, on, on, on};
          const int exp = vector_exponent(y, counts, lanes);
          const float f = pow2(-exp);
          if (on)
            *reinterpret_cast<uint2*>(out + u * each * out_step) =
                make_uint2(e4m3x2(y[0] * f, y[1] * f) | e4m3x2(y[2] * f, y[3] * f) << 16,
                           e4m3x2(y[4] * f, y[5] * f) | e4m3x2(y[6] * f, y[7] * f) << 16);
          if (on && c == 0) exps[u * each * e_step] = static_cast<int8_t>(exp);
        } else if (on) {
          if constexpr (decltype(rotate)::value) {
            if (turned) raw[u].set(y);
          }
          raw[u].store(out + u * each * out_step);
        }
      }
      in += kRopeFlight * each * step, out += kRopeFlight * each * out_step, exps += kRopeFlight * each * e_step;
    }
  };
  constexpr Yes yes;
  constexpr No no;
  if (a.heads > 0) {
    if (a.half > 0)
      heads(yes, no, a.q + row * a.q_row, a.q_head, a.heads, a.oq + row * a.oq_row, a.oq_head, nullptr, 0);
    else
      heads(no, no, a.q + row * a.q_row, a.q_head, a.heads, a.oq + row * a.oq_row, a.oq_head, nullptr, 0);
  }
  if (a.kv_heads == 0) return;
  const int64_t slot = __ldg(a.slots + row);
  if (slot >= a.n_slots && lane == 0 && a.dev_error != nullptr) atomicOr(a.dev_error, SV_DEVERR_PAGE);
  if (slot < 0 || slot >= a.n_slots) return;
  const int64_t b = slot <= INT32_MAX ? a.by_page.of(static_cast<int>(slot)) : slot / a.page;
  const int64_t t = slot - b * a.page, at = b * a.block + t * a.token, e_at = b * a.e_block + t * a.e_token;
  const std::conditional_t<QUANT, Yes, No> codes;
  if (a.half > 0)
    heads(yes, codes, a.k + row * a.k_row, a.k_head, a.kv_heads, a.k_cache + at, a.head, a.k_exps + e_at, a.e_head);
  else
    heads(no, codes, a.k + row * a.k_row, a.k_head, a.kv_heads, a.k_cache + at, a.head, a.k_exps + e_at, a.e_head);
  heads(no, codes, a.v + row * a.v_row, a.v_head, a.kv_heads, a.v_cache + at, a.head, a.v_exps + e_at, a.e_head);
}

// A group of lanes a vector.  WIDE: every vector starts on 16 bytes, dimensions and
// pairs are whole chunks of eight; otherwise elements are loaded one by one.  QUANT: the
// caches hold e4m3 and exponents.
template <typename T, bool QUANT, bool PAIRS, bool WIDE>
__global__ __launch_bounds__(kRopeThreads) void rope_kernel(const __grid_constant__ RopeArgs a) {
  extern __shared__ __align__(16) float4 sines[];  // two pairs' (cos, sin) a unit
  const int tid = threadIdx.x, lane = tid & 31;
  const int lanes = 1 << a.lanes_log2, c = tid & (lanes - 1), group = tid >> a.lanes_log2;
  const int groups = kRopeThreads >> a.lanes_log2;
  const int block = static_cast<int>(blockIdx.x);
  const bool query = block < a.q_ctas, value = block >= a.q_ctas + a.kv_ctas;
  const int heads = query ? a.heads : a.kv_heads, total = a.n_rows * heads;
  const FastDiv by_heads = query ? a.by_heads : a.by_kv_heads;
  const char* const in = query ? a.q : value ? a.v : a.k;
  const int64_t in_row = query ? a.q_row : value ? a.v_row : a.k_row,
                in_head = query ? a.q_head : value ? a.v_head : a.k_head;
  const int first = (block - (query ? 0 : value ? a.q_ctas + a.kv_ctas : a.q_ctas)) * groups;
  const int end = min(first + groups, total);
  const int row0 = by_heads.of(first), rows = by_heads.of(end - 1) - row0 + 1;
  const int d0 = c * 8, half = a.half;
  const bool mine = d0 < a.dim;

  // the vector, and where it goes
  const int at = first + group;
  const bool some = at < end;
  const int row = some ? by_heads.of(at) : row0, h = some ? at - row * heads : 0;
  const char* const src = in + row * in_row + h * in_head;
  char* to = nullptr;  // NULL: nowhere
  int8_t* exps = nullptr;
  Eight<T> raw;
  float y[8], other[8];  // not WIDE: the elements and their partners
  if constexpr (WIDE) {
    if (some && mine) raw.load(src + d0 * sizeof(T));
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int d = d0 + e;
      const int p = PAIRS ? d ^ 1 : d < half ? d + half : d - half;
      y[e] = some && d < a.dim ? to_float(reinterpret_cast<const T*>(src)[d]) : 0.0f;
      other[e] = some && d < 2 * half ? to_float(reinterpret_cast<const T*>(src)[p]) : 0.0f;
    }
  }
  if (some && query) {
    to = a.oq + row * a.oq_row + h * a.oq_head;
  } else if (some) {
    const int64_t slot = __ldg(a.slots + row);
    if (slot >= a.n_slots && a.dev_error != nullptr) atomicOr(a.dev_error, SV_DEVERR_PAGE);
    if (slot >= 0 && slot < a.n_slots) {
      const int64_t b = slot <= INT32_MAX ? a.by_page.of(static_cast<int>(slot)) : slot / a.page;
      const int64_t t = slot - b * a.page;
      to = (value ? a.v_cache : a.k_cache) + b * a.block + t * a.token + h * a.head;
      if constexpr (QUANT)
        exps = (value ? a.v_exps : a.k_exps) + b * a.e_block + t * a.e_token + h * a.e_head;
    }
  }

  const bool turned = !value && d0 < 2 * half;
  if constexpr (WIDE) raw.get(y);
  if (!value && half > 0) {  // the CTA's rows' sines
    for (int i = tid; i < rows * half; i += kRopeThreads) {
      const int r = a.by_half.of(i), f = i - r * half;
      reinterpret_cast<float2*>(sines)[r * padded_pairs(half) + (WIDE ? sine_place(f) : f)] =
          sine_of(__ldg(a.positions + row0 + r), __ldg(a.freqs + f), a.amplitude);
    }
    __syncthreads();
    if constexpr (WIDE) {
      float co[8], si[8];
      if (turned) lane_sines<PAIRS>(sines + (row - row0) * (padded_pairs(half) >> 1), d0, half, co, si);
      turn_chunk<T, PAIRS>(raw, partners_of(lane, c, half), turned, co, si, y);
    } else {
      const float2* const mine_sines = reinterpret_cast<const float2*>(sines) + (row - row0) * padded_pairs(half);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int d = d0 + e;
        if (d >= 2 * half) continue;
        const float2 z = mine_sines[PAIRS ? d >> 1 : d < half ? d : d - half];
        y[e] = y[e] * z.x + other[e] * ((PAIRS ? d & 1 : d >= half) ? z.y : -z.y);
      }
    }
  }
  if (!QUANT || query) {
    if (to == nullptr || !mine) return;
    if constexpr (WIDE) {
      if (turned) raw.set(y);
      raw.store(to + d0 * sizeof(T));
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (d0 + e < a.dim) reinterpret_cast<T*>(to)[d0 + e] = from_float<T>(y[e]);
    }
    return;
  }
  if constexpr (QUANT) {
    bool counts[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) counts[e] = some && d0 + e < a.dim;
    const int exp = vector_exponent(y, counts, lanes);
    if (to == nullptr) return;
    const float f = pow2(-exp);
    if constexpr (WIDE) {
      if (mine)
        *reinterpret_cast<uint2*>(to + d0) =
            make_uint2(e4m3x2(y[0] * f, y[1] * f) | e4m3x2(y[2] * f, y[3] * f) << 16,
                       e4m3x2(y[4] * f, y[5] * f) | e4m3x2(y[6] * f, y[7] * f) << 16);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (d0 + e < a.dim) to[d0 + e] = static_cast<char>(e4m3x2(y[e] * f, 0.0f));
    }
    if (c == 0) *exps = static_cast<int8_t>(exp);
  }
}

template <typename T, bool QUANT, bool PAIRS>
int launch_rope(const RopeArgs& args, bool wide, int sms, cudaStream_t st) {
  RopeArgs a = args;
  constexpr int kWarps = kRopeThreads / 32;
  // rows for eight warps of every SM.  At 608 / 1,216 / 2,432 rows a warp a row and a group a
  // vector take, of 32/8 heads of 128 into 8 bits, 7.7 and 6.5 / 8.0 and 11.2 / 9.8 and 20.3
  // us; of 16/4 heads of 80 into bf16 5.3 and 3.7 / 5.3 and 5.7 / 6.0 and 9.5; of 8/1 heads
  // of 64 3.5 and 3.0 / 3.5 and 3.3 / 3.8 and 4.0
  if (wide && a.n_rows >= kWarps * sms)
    return launch(rope_row_kernel<T, QUANT, PAIRS>, dim3((a.n_rows + kWarps - 1) / kWarps), kRopeThreads,
                  kWarps * padded_pairs(a.half) * static_cast<int>(sizeof(float2)), 1, false, st, a);
  const int groups = kRopeThreads >> a.lanes_log2;
  auto ctas = [&](int heads) { return (a.n_rows * heads + groups - 1) / groups; };
  a.q_ctas = ctas(a.heads), a.kv_ctas = ctas(a.kv_heads);
  const int smem = std::max(a.heads > 0 ? rope_smem(groups, a.heads, a.half) : 0,
                            a.kv_heads > 0 ? rope_smem(groups, a.kv_heads, a.half) : 0);
  const dim3 grid(static_cast<unsigned>(a.q_ctas + 2 * a.kv_ctas));
  return wide ? launch(rope_kernel<T, QUANT, PAIRS, true>, grid, kRopeThreads, smem, 1, false, st, a)
              : launch(rope_kernel<T, QUANT, PAIRS, false>, grid, kRopeThreads, smem, 1, false, st, a);
}

template <typename T>
int pick_rope(const RopeArgs& a, bool quant, bool pairs, bool wide, int sms, cudaStream_t st) {
  if (quant)
    return pairs ? launch_rope<T, true, true>(a, wide, sms, st) : launch_rope<T, true, false>(a, wide, sms, st);
  return pairs ? launch_rope<T, false, true>(a, wide, sms, st) : launch_rope<T, false, false>(a, wide, sms, st);
}

}  // namespace
}  // namespace serve
}  // namespace sv

extern "C" {

int spec_verify_rope_append(const void* query, int64_t q_row_stride, int64_t q_head_stride,
                            int32_t heads, const void* key, const void* value,
                            int64_t k_row_stride, int64_t k_head_stride, int64_t v_row_stride,
                            int64_t v_head_stride, int32_t kv_heads, int32_t n_rows,
                            int32_t head_dim, int32_t dtype, const int32_t* positions,
                            const int64_t* freqs, int32_t rotary_dim, int32_t interleaved,
                            float amplitude, void* out_query, int64_t oq_row_stride,
                            int64_t oq_head_stride, const int64_t* slots, void* key_cache,
                            void* value_cache, int64_t block_stride, int64_t token_stride,
                            int64_t head_stride, int32_t num_blocks, int32_t page_size,
                            int32_t cache_dtype, int8_t* key_exps, int8_t* value_exps,
                            int64_t e_block_stride, int64_t e_token_stride, int64_t e_head_stride,
                            int32_t* dev_error, void* stream) {
  using namespace sv::serve;
  if (dtype != SV_BF16 && dtype != SV_FP32) return SV_ERR_DTYPE;
  if (kv_heads > 0 && cache_dtype != dtype && cache_dtype != SV_E4M3) return SV_ERR_DTYPE;
  const int es = dtype == SV_BF16 ? 2 : 4;
  const bool quant = kv_heads > 0 && cache_dtype == SV_E4M3;
  if (heads < 0 || kv_heads < 0 || heads + static_cast<int64_t>(kv_heads) < 1 || n_rows < 0 ||
      head_dim < 1 || rotary_dim < 0 || rotary_dim > head_dim || rotary_dim % 2 != 0 ||
      !std::isfinite(amplitude))
    return SV_ERR_ARG;
  if (kv_heads > 0 && (num_blocks < 1 || page_size < 1)) return SV_ERR_ARG;
  if (head_dim > SV_ATTN_MAX_HEAD_DIM) return SV_ERR_UNSUPPORTED;
  const int64_t total = n_rows * (heads + 2 * static_cast<int64_t>(kv_heads));
  if (heads > (1 << 20) || kv_heads > (1 << 20) || total > INT32_MAX / 2) return SV_ERR_UNSUPPORTED;
  if (n_rows == 0) return SV_OK;  // an empty tensor has no address
  if (heads > 0 && (query == nullptr || out_query == nullptr)) return SV_ERR_ARG;
  if (kv_heads > 0 && (key == nullptr || value == nullptr || slots == nullptr ||
                       key_cache == nullptr || value_cache == nullptr))
    return SV_ERR_ARG;
  if (quant && (key_exps == nullptr || value_exps == nullptr)) return SV_ERR_ARG;
  if (rotary_dim > 0 && (positions == nullptr || freqs == nullptr)) return SV_ERR_ARG;
  if (!aligned_to(positions, 4) || !aligned_to(freqs, 8) || !aligned_to(slots, 8) ||
      !null_or_aligned(dev_error, 4))
    return SV_ERR_ARG;
  if (heads == 0) query = nullptr, out_query = nullptr, q_row_stride = q_head_stride = oq_row_stride = oq_head_stride = 0;
  if (kv_heads == 0) {
    key = value = nullptr, key_cache = value_cache = nullptr, slots = nullptr;
    k_row_stride = k_head_stride = v_row_stride = v_head_stride = 0;
    block_stride = token_stride = head_stride = 0, page_size = num_blocks = 1;
  }
  if (!quant) key_exps = value_exps = nullptr, e_block_stride = e_token_stride = e_head_stride = 0;
  uint64_t in = 0, cache = 0;
  for (const void* p : {query, key, value, static_cast<const void*>(out_query)})
    in |= reinterpret_cast<uint64_t>(p);
  for (int64_t s : {q_row_stride, q_head_stride, k_row_stride, k_head_stride, v_row_stride,
                    v_head_stride, oq_row_stride, oq_head_stride}) {
    if (s < 0) return SV_ERR_ARG;
    in |= static_cast<uint64_t>(s) * es;
  }
  const int cs = quant ? 1 : es;
  cache |= reinterpret_cast<uint64_t>(key_cache) | reinterpret_cast<uint64_t>(value_cache);
  for (int64_t s : {block_stride, token_stride, head_stride}) {
    if (s < 0) return SV_ERR_ARG;
    cache |= static_cast<uint64_t>(s) * cs;
  }
  if (e_block_stride < 0 || e_token_stride < 0 || e_head_stride < 0) return SV_ERR_ARG;
  if (in % es != 0 || cache % cs != 0) return SV_ERR_ARG;
  const bool pairs = interleaved != 0;
  const bool wide = in % 16 == 0 && cache % (quant ? 8 : 16) == 0 && head_dim % 8 == 0 &&
                    rotary_dim % 8 == 0;
  Device d;
  const int rc = device(&d);
  if (rc != SV_OK) return rc;
  const int half = rotary_dim / 2;
  RopeArgs a{static_cast<const char*>(query), static_cast<const char*>(key),
             static_cast<const char*>(value), q_row_stride * es, q_head_stride * es,
             k_row_stride * es, k_head_stride * es, v_row_stride * es, v_head_stride * es,
             static_cast<char*>(out_query), oq_row_stride * es, oq_head_stride * es, positions,
             freqs, slots, static_cast<char*>(key_cache), static_cast<char*>(value_cache),
             block_stride * cs, token_stride * cs, head_stride * cs, key_exps, value_exps,
             e_block_stride, e_token_stride, e_head_stride,
             static_cast<int64_t>(num_blocks) * page_size, dev_error, n_rows, heads, kv_heads,
             head_dim, half, 0, 0, page_size, head_dim <= 64 ? 3 : head_dim <= 128 ? 4 : 5,
             amplitude, FastDiv::by(static_cast<uint32_t>(std::max(heads, 1))),
             FastDiv::by(static_cast<uint32_t>(std::max(kv_heads, 1))),
             FastDiv::by(static_cast<uint32_t>(std::max(half, 1))),
             FastDiv::by(static_cast<uint32_t>(page_size))};
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return dtype == SV_BF16 ? pick_rope<__nv_bfloat16>(a, quant, pairs, wide, d.sms, st)
                          : pick_rope<float>(a, quant, pairs, wide, d.sms, st);
}

int spec_verify_rope(const void* x, int64_t row_stride, int64_t x_head_stride, int32_t n_rows,
                     int32_t heads, int32_t head_dim, int32_t dtype, const int32_t* positions,
                     const int64_t* freqs, int32_t rotary_dim, int32_t interleaved,
                     float amplitude, void* out, int64_t out_row_stride, int64_t out_head_stride,
                     void* stream) {
  if (heads < 1) return SV_ERR_ARG;
  return spec_verify_rope_append(x, row_stride, x_head_stride, heads, nullptr, nullptr, 0, 0, 0, 0,
                                 0, n_rows, head_dim, dtype, positions, freqs, rotary_dim,
                                 interleaved, amplitude, out, out_row_stride, out_head_stride,
                                 nullptr, nullptr, nullptr, 0, 0, 0, 0, 0, dtype, nullptr, nullptr,
                                 0, 0, 0, nullptr, stream);
}

}  // extern "C"
