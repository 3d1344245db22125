// sv_attn_fma.cuh -- attention in fp32 (the tensor cores have no product that
// keeps 24 bits).
//
// Rows are packed and work is split as in the tensor core kernel, with items of 32
// rows: four warps of eight rows.  32 keys at a time lie in shared memory (two
// buffers, filled ahead by 16-byte copies): for the scores a lane holds a key and
// eight accumulators, for the weighted sum of the values it holds every 32nd
// quartet of the head's dimensions.  Bound by shared memory reads: 12 wavefronts
// of K and Q beside 32 FMAs a warp and four dimensions.  32 requests of 16 tokens,
// 32 heads over 8 of 128, 4,096 cached: 1.51 ms (22.9 TFLOP/s); with one warp a row
// and no sharing of keys it was 11.7 ms.  8 single tokens, 8 heads of 64, 2,048
// cached: 69 us, and 658 us without the split over keys.  A row alone in its item
// pays for its warp's other seven.
#pragma once

#include "sv_attn_mma.cuh"

namespace sv {
namespace serve {

constexpr int kFmaRows = 32, kFmaKeys = 32, kFmaThreads = 128, kFmaWarpRows = 8;

constexpr int kFmaWeights = kFmaRows + 4;  // floats a key; padded against bank conflicts

__host__ __device__ constexpr int fma_row(int dp) { return dp + 4; }  // of a key, likewise
__host__ __device__ constexpr int fma_smem(int dp) {
  return (kFmaRows * dp + 2 * kFmaKeys * (fma_row(dp) + dp) + kFmaKeys * kFmaWeights) * 4 + 256;
}

template <int DP>
__global__ __launch_bounds__(kFmaThreads) void attn_fma_kernel(const MmaArgs p) {
  constexpr int MR = kFmaRows, KR = fma_row(DP);
  constexpr int kVec = DP / 32 >= 4 ? 4 : 2, kSets = DP / 32 / kVec;  // dimensions of a lane
  extern __shared__ __align__(16) float fsm[];
  float* const qs = fsm;                              // [MR][DP]
  float* const ks = qs + MR * DP;                     // [2][32][KR]
  float* const vs = ks + 2 * kFmaKeys * KR;           // [2][32][DP]
  float* const ps = vs + 2 * kFmaKeys * DP;           // [32 keys][kFmaWeights]
  const AttnArgs& a = p.a;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  Walk<MR> walk;
  static_assert(sizeof(PlanSmem<MR>) <= 256, "plan block");
  const bool any = plan<MR, kFmaThreads>(
      p, reinterpret_cast<PlanSmem<MR>*>(ps + kFmaKeys * kFmaWeights), &walk);
  grid_dep_launch_dependents();
  if (!any) return;
  uint32_t err = 0;
  Segment g;
  while (walk.next(p, &g)) {
    const int32_t* table = a.table + g.r * a.table_stride;
    const int first = g.tile0 * kTile, last = min(g.tile1 * kTile, g.kv_end);
    const int steps = max(1, (last - first + kFmaKeys - 1) / kFmaKeys);
    __syncthreads();  // the segment before is done with shared memory
    for (int i = tid; i < MR * (DP / 4); i += kFmaThreads) {
      const int row = i / (DP / 4), d = i % (DP / 4) * 4, x = g.m * MR + row;
      const bool on = row < g.rows && d < a.dim;
      const int j = a.by_group.of(x);
      const char* src = a.q + static_cast<int64_t>(g.row0 + j) * a.q_row +
                        static_cast<int64_t>(g.h * a.group + x - j * a.group) * a.q_head;
      cp_async16(smem_addr(qs + row * DP + d), on ? src + d * 4 : a.q, on ? 16 : 0);
    }
    auto fetch = [&](int step) {  // keys first + 32 step ..: a warp eight of them
      if (step < steps)
        for (int r = warp; r < kFmaKeys; r += kFmaThreads / 32) {
          const int t = first + step * kFmaKeys + r;
          int64_t at = -1;
          if (t < last) {
            const int page = a.by_page.of(t);
            int id = __ldg(table + page);
            if (id < 0 || id >= a.num_blocks) err |= SV_DEVERR_PAGE, id = 0;
            at = id * a.block + (t - page * a.page) * a.token + g.h * a.head;
          }
          for (int d = lane * 4; d < DP; d += 128) {
            const bool on = at >= 0 && d < a.dim;
            cp_async16(smem_addr(ks + ((step & 1) * kFmaKeys + r) * KR + d),
                       on ? a.k + at + d * 4 : a.k, on ? 16 : 0);
            cp_async16(smem_addr(vs + ((step & 1) * kFmaKeys + r) * DP + d),
                       on ? a.v + at + d * 4 : a.v, on ? 16 : 0);
          }
        }
      cp_async_commit();
    };
    // the warp's rows
    int pos[kFmaWarpRows], lo[kFmaWarpRows];
    float m[kFmaWarpRows], l[kFmaWarpRows], o[kFmaWarpRows][kSets * kVec];
#pragma unroll
    for (int r = 0; r < kFmaWarpRows; ++r) {
      pos[r] = g.seq - g.l + a.by_group.of(g.m * MR + warp * kFmaWarpRows + r);
      lo[r] = a.window > 0 ? max(0, pos[r] - a.window + 1) : 0;
      m[r] = -kInf, l[r] = 0.0f;
#pragma unroll
      for (int d = 0; d < kSets * kVec; ++d) o[r][d] = 0.0f;
    }
    const int rows = g.rows - warp * kFmaWarpRows;  // of this warp
    const int all_hi = pos[0] + 1, all_lo = lo[kFmaWarpRows - 1];
    fetch(0);
    for (int step = 0; step < steps; ++step) {
      fetch(step + 1);
      cp_async_wait<1>();
      __syncthreads();
      const int t0 = first + step * kFmaKeys;
      const float* k = ks + ((step & 1) * kFmaKeys + lane) * KR;
      const float* v = vs + (step & 1) * kFmaKeys * DP;
      if (rows > 0) {
        const bool edge = t0 + kFmaKeys > all_hi || t0 < all_lo || t0 + kFmaKeys > last;
        float s[kFmaWarpRows];
#pragma unroll
        for (int r = 0; r < kFmaWarpRows; ++r) s[r] = 0.0f;
#pragma unroll 4
        for (int d = 0; d < DP; d += 4) {
          const float4 x = *reinterpret_cast<const float4*>(k + d);
#pragma unroll
          for (int r = 0; r < kFmaWarpRows; ++r) {
            const float4 y =
                *reinterpret_cast<const float4*>(qs + (warp * kFmaWarpRows + r) * DP + d);
            s[r] = fmaf(x.x, y.x, s[r]), s[r] = fmaf(x.y, y.y, s[r]);
            s[r] = fmaf(x.z, y.z, s[r]), s[r] = fmaf(x.w, y.w, s[r]);
          }
        }
        const int t = t0 + lane;
        float* const pw = ps + lane * kFmaWeights + warp * kFmaWarpRows;
        float w[kFmaWarpRows];
#pragma unroll
        for (int r = 0; r < kFmaWarpRows; ++r) {
          s[r] *= a.scale2;
          if (edge && !(t < last && t <= pos[r] && t >= lo[r])) s[r] = -kInf;
          float top = s[r];
#pragma unroll
          for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, d));
          top = fmaxf(top, m[r]);
          const float base = top == -kInf ? 0.0f : top, keep = ex2(m[r] - base);
          w[r] = ex2(s[r] - base);
          l[r] = l[r] * keep + w[r];
          m[r] = top;
#pragma unroll
          for (int d = 0; d < kSets * kVec; ++d) o[r][d] *= keep;
        }
        *reinterpret_cast<float4*>(pw) = make_float4(w[0], w[1], w[2], w[3]);
        *reinterpret_cast<float4*>(pw + 4) = make_float4(w[4], w[5], w[6], w[7]);
        __syncwarp();
        const int n = min(kFmaKeys, last - t0);
        for (int j = 0; j < n; ++j) {
          const float* pj = ps + j * kFmaWeights + warp * kFmaWarpRows;
          const float4 x = *reinterpret_cast<const float4*>(pj),
                       y = *reinterpret_cast<const float4*>(pj + 4);
          float pr[kFmaWarpRows] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
          float e[kSets * kVec];
#pragma unroll
          for (int i = 0; i < kSets; ++i) {
            const float* at = v + j * DP + (i * 32 + lane) * kVec;
            if constexpr (kVec == 4) {
              const float4 z = *reinterpret_cast<const float4*>(at);
              e[i * 4] = z.x, e[i * 4 + 1] = z.y, e[i * 4 + 2] = z.z, e[i * 4 + 3] = z.w;
            } else {
              const float2 z = *reinterpret_cast<const float2*>(at);
              e[i * 2] = z.x, e[i * 2 + 1] = z.y;
            }
          }
          if (edge) {  // a value that a row does not see stays out, whatever it is
#pragma unroll
            for (int r = 0; r < kFmaWarpRows; ++r)
              if (t0 + j <= pos[r] && t0 + j >= lo[r]) {
#pragma unroll
                for (int d = 0; d < kSets * kVec; ++d) o[r][d] = fmaf(pr[r], e[d], o[r][d]);
              }
          } else {
#pragma unroll
            for (int r = 0; r < kFmaWarpRows; ++r)
#pragma unroll
              for (int d = 0; d < kSets * kVec; ++d) o[r][d] = fmaf(pr[r], e[d], o[r][d]);
          }
        }
      }
      __syncthreads();  // this buffer and the weights may be written again
    }
    const int slot = 2 * blockIdx.x + (g.begins ? 1 : 0);
#pragma unroll
    for (int r = 0; r < kFmaWarpRows; ++r) {
      if (r >= rows) break;
      float z = l[r];
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) z += __shfl_xor_sync(~0u, z, d);
      const int prow = warp * kFmaWarpRows + r, x = g.m * MR + prow;
      const int64_t orow = g.row0 + a.by_group.of(x);
      const int head = g.h * a.group + x - a.by_group.of(x) * a.group;
      const float inv = g.whole ? (z > 0.0f || z != z ? 1.0f / z : 0.0f) : 1.0f;
#pragma unroll
      for (int i = 0; i < kSets; ++i)
#pragma unroll
        for (int c = 0; c < kVec; ++c) {
          const int d = (i * 32 + lane) * kVec + c;
          if (d >= a.dim) continue;
          if (g.whole)
            reinterpret_cast<float*>(a.out + orow * a.o_row + head * a.o_head)[d] =
                o[r][i * kVec + c] * inv;
          else
            reinterpret_cast<float*>(
                p.o + (static_cast<int64_t>(slot) * (DP / 4) + d / 4) * MR + prow)[d % 4] =
                o[r][i * kVec + c];
        }
      if (lane == 0) {
        if (!g.whole)
          p.ml[static_cast<int64_t>(slot) * MR + prow] = make_float2(m[r], z);
        else if (a.lse != nullptr)
          a.lse[orow * a.heads + head] = z > 0.0f || z != z ? (m[r] + log2f(z)) * kLn2 : -kInf;
      }
    }
  }
  if (err != 0 && a.dev_error != nullptr) atomicOr(a.dev_error, static_cast<int32_t>(err));
}

}  // namespace serve
}  // namespace sv
