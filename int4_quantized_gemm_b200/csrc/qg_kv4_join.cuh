// qg_kv4_join.cuh -- joining the parts of attention rows whose keys several
// workers took: sum_i 2^(m_i - m) (l_i, o_i), m the largest m_i.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "qg_kv4.cuh"

namespace qg {

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ uint32_t half2_bits(float lo, float hi) {
  __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&h);
}

// Adds `count` parts of a row, a warp: the log2 maximum and the sum p of part i at head(i), its dim sums p v at
// sums(i); their total's maximum and sum, and D / 32 values in each lane.  The parts' weights first, a lane each: no
// load waits for another part's.
template <int D, class F, class H>
__device__ __forceinline__ void add_parts(F sums, H head, int count, int lane, float& top, float& l,
                                          float (&v)[D / 32]) {
  constexpr int V = D / 32, kBatch = 8;
  top = -INFINITY;
  l = 0.0f;
#pragma unroll
  for (int k = 0; k < V; ++k) v[k] = 0.0f;
#pragma unroll 1
  for (int i0 = 0; i0 < count; i0 += 32) {
    const int n = min(32, count - i0);
    float x[kBatch][V];
    const auto load = [&](int i) {
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
#pragma unroll
        for (int k = 0; k < V; ++k) x[b][k] = 0.0f;
        if (i + b < n) {
          const float* p = sums(i0 + i + b) + V * lane;
          if constexpr (V == 4) *reinterpret_cast<float4*>(x[b]) = *reinterpret_cast<const float4*>(p);
          else *reinterpret_cast<float2*>(x[b]) = *reinterpret_cast<const float2*>(p);
        }
      }
    };
    float2 ml = make_float2(-INFINITY, 0.0f);
    if (lane < n) ml = *head(i0 + lane);
    load(0);
    float t = ml.x;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, d));
    t = fmaxf(t, top);
    const float safe = t == -INFINITY ? 0.0f : t;
    const float f = ex2(top - safe), g = ex2(ml.x - safe);
    float sum = ml.y * g;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
    l = fmaf(l, f, sum);
    top = t;
#pragma unroll
    for (int k = 0; k < V; ++k) v[k] *= f;
#pragma unroll 1
    for (int i = 0;;) {
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        const float gb = __shfl_sync(0xffffffffu, g, (i + b) & 31);
#pragma unroll
        for (int k = 0; k < V; ++k) v[k] = fmaf(x[b][k], i + b < n ? gb : 0.0f, v[k]);
      }
      i += kBatch;
      if (i >= n) break;
      load(i);
    }
  }
}

// out (and lse) of a row of an item from its sums, a warp
template <int D>
__device__ __forceinline__ void write_row(const Attn4& a, int first, int h, int row, int lane, float top, float l,
                                          const float (&v)[D / 32]) {
  constexpr int V = D / 32;
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
  const int t = first + row / a.group, hq = h * a.group + row % a.group;
  uint32_t b[V / 2];
#pragma unroll
  for (int i = 0; i < V / 2; ++i) {
    const float x = l == 0.0f ? 0.0f : v[2 * i] * inv, y = l == 0.0f ? 0.0f : v[2 * i + 1] * inv;
    if (a.dtype == QG_F16) {
      b[i] = half2_bits(x, y);
    } else {
      __nv_bfloat162 hv = __floats2bfloat162_rn(x, y);
      b[i] = *reinterpret_cast<uint32_t*>(&hv);
    }
  }
  char* p = static_cast<char*>(a.out) + 2 * (t * a.o_st + hq * a.o_sh + V * lane);
  if constexpr (V == 4) *reinterpret_cast<uint2*>(p) = make_uint2(b[0], b[1]);
  else *reinterpret_cast<uint32_t*>(p) = b[0];
  if (a.lse && lane == 0) a.lse[(int64_t)t * a.heads_q + hq] = l == 0.0f ? -INFINITY : (top + log2f(l)) * 0.69314718056f;
}

}  // namespace qg
