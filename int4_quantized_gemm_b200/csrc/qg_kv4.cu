// qg_kv4.cu -- quantizing keys and values into the paged 4-bit cache as they
// are written, and reading tokens back (layout: qg_kv4.cuh).
//
// For each group of 64 channels (binary32, then fp16 where held):
//   lo, hi = min, max of the group, its values x held to +-65504
//   s = fp16(max((hi - lo) / 15, 1e-5)),  o = fp16(lo)
//   q = clamp(rint((x - o) / s), 0, 15)
// with the rounded s and o, so a code is the nearest one for the values that
// will be read.  A NaN in the group makes s and o NaN (and its codes 0).
//
// Both kernels are memory-bound: 2 + 9/16 bytes per value (a value, its code,
// 1/64 of its group's params).  One thread owns one word (8 channels, one
// 16-byte access of the 16-bit side); a group is 8 consecutive lanes.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "qg_device.cuh"
#include "qg_internal.h"
#include "qg_kv4.cuh"

namespace qg {

static __device__ unsigned long long g_status_kv4;

unsigned long long read_clear_status_kv4(cudaStream_t s) {
  unsigned long long v = 0, z = 0;
  cudaMemcpyFromSymbolAsync(&v, g_status_kv4, sizeof(v), 0, cudaMemcpyDeviceToHost, s);
  cudaMemcpyToSymbolAsync(g_status_kv4, &z, sizeof(z), 0, cudaMemcpyHostToDevice, s);
  cudaStreamSynchronize(s);
  return v;
}

namespace {

__device__ __forceinline__ void report_slot() {
  atomicCAS(&g_status_kv4, 0ull,
            (unsigned long long)kDevBadArg | (1ull << 8) | ((unsigned long long)blockIdx.x << 24));
}

template <typename T>
struct Pair;
template <>
struct Pair<__half> {
  using V = __half2;
  static __device__ __forceinline__ float2 f32(V v) { return __half22float2(v); }
  static __device__ __forceinline__ V round(float a, float b) { return __floats2half2_rn(a, b); }
};
template <>
struct Pair<__nv_bfloat16> {
  using V = __nv_bfloat162;
  static __device__ __forceinline__ float2 f32(V v) { return __bfloat1622float2(v); }
  static __device__ __forceinline__ V round(float a, float b) { return __floats2bfloat162_rn(a, b); }
};

__device__ __forceinline__ float min_nan(float a, float b) {
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

struct KVIn {
  const void* p[2];
  int64_t st[2], sh[2];  // token and head strides (elements)
};

// Codes of 8 values against scale s and offset o.  The quotient is first taken
// with 1/s; rounding differs from the division's only next to a half-integer,
// where the group of 8 is done again with the division.
__device__ __forceinline__ uint32_t codes8(const float (&x)[8], float s, float o) {
  const float inv = __fdiv_rn(1.0f, s);
  uint32_t w = 0;
  bool near_tie = false;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float t = __fmul_rn(__fsub_rn(x[i], o), inv);
    const float c = fminf(fmaxf(t, 0.0f), 15.0f);  // NaN: 0
    const float q = rintf(c);
    near_tie |= fabsf(c - q) > 0.4999f;
    w |= (uint32_t)q << (4 * i);
  }
  if (near_tie) {
    w = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float t = __fdiv_rn(__fsub_rn(x[i], o), s);
      w |= (uint32_t)rintf(fminf(fmaxf(t, 0.0f), 15.0f)) << (4 * i);
    }
  }
  return w;
}

template <typename T>
__global__ void __launch_bounds__(256)
    quantize_kv4_kernel(KVIn in, const int64_t* __restrict__ slots, KV4 cache, int64_t words, int words_per_token) {
  pdl_trigger();
  pdl_wait();
  const int groups = cache.dim / 64;
  const int64_t limit = cache.pages * cache.page_size;
  // `words` is a multiple of 8 and so is the stride: a group's 8 lanes stay together
  for (int64_t u = (int64_t)blockIdx.x * 256 + threadIdx.x; u < words; u += (int64_t)gridDim.x * 256) {
    const int64_t token = u / (2 * words_per_token);
    int w = (int)(u - token * (2 * words_per_token));
    const int kv = w >= words_per_token;
    w -= kv * words_per_token;
    const int j = w & 7, g = (w >> 3) % groups, h = (w >> 3) / groups;
    const int64_t slot = __ldg(slots + token);
    if (slot < 0 || slot >= limit) {  // the same for the group's 8 lanes
      if (slot >= limit) report_slot();
      continue;
    }
    const T* src = static_cast<const T*>(in.p[kv]) + token * in.st[kv] + h * in.sh[kv] + 64 * g + 8 * j;
    const uint4 raw = *reinterpret_cast<const uint4*>(src);
    float x[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = Pair<T>::f32(reinterpret_cast<const typename Pair<T>::V*>(&raw)[i]);
      x[2 * i] = min_nan(max_nan(f.x, -65504.0f), 65504.0f);
      x[2 * i + 1] = min_nan(max_nan(f.y, -65504.0f), 65504.0f);
    }
    float lo = x[0], hi = x[0];
#pragma unroll
    for (int i = 1; i < 8; ++i) {
      lo = min_nan(lo, x[i]);
      hi = max_nan(hi, x[i]);
    }
    const uint32_t mask = 0xFFu << (threadIdx.x & 24);
#pragma unroll
    for (int d = 4; d > 0; d >>= 1) {
      lo = min_nan(lo, __shfl_xor_sync(mask, lo, d));
      hi = max_nan(hi, __shfl_xor_sync(mask, hi, d));
    }
    const __half2 so = __floats2half2_rn(max_nan(__fdiv_rn(__fsub_rn(hi, lo), 15.0f), 1e-5f), lo);
    const float2 f = __half22float2(so);
    const int64_t page = slot / cache.page_size;
    const int64_t row = kv4_row(cache, page, h) + (slot - page * cache.page_size);
    cache.codes[kv][(row * 8 + j) * groups + g] = codes8(x, f.x, f.y);
    if (j == 0) cache.params[kv][row * groups + g] = *reinterpret_cast<const uint32_t*>(&so);
  }
}

template <typename T>
__device__ __forceinline__ void put8(T* p, const float (&x)[8]) {
  typename Pair<T>::V o[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) o[i] = Pair<T>::round(x[2 * i], x[2 * i + 1]);
  *reinterpret_cast<uint4*>(p) = *reinterpret_cast<uint4*>(o);
}
template <>
__device__ __forceinline__ void put8<float>(float* p, const float (&x)[8]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
}

struct KVOut {
  void* p[2];
  int64_t st[2], sh[2];
};

template <typename T>
__global__ void __launch_bounds__(256)
    dequantize_kv4_kernel(KVOut out, const int64_t* __restrict__ slots, KV4 cache, int64_t words,
                          int words_per_token) {
  pdl_trigger();
  pdl_wait();
  const int groups = cache.dim / 64;
  const int64_t limit = cache.pages * cache.page_size;
  for (int64_t u = (int64_t)blockIdx.x * 256 + threadIdx.x; u < words; u += (int64_t)gridDim.x * 256) {
    const int64_t token = u / (2 * words_per_token);
    int w = (int)(u - token * (2 * words_per_token));
    const int kv = w >= words_per_token;
    w -= kv * words_per_token;
    const int j = w & 7, g = (w >> 3) % groups, h = (w >> 3) / groups;
    const int64_t slot = __ldg(slots + token);
    float x[8];
    if (slot < 0 || slot >= limit) {
      if (slot >= limit) report_slot();
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = 0.0f;
    } else {
      const int64_t page = slot / cache.page_size;
      const int64_t row = kv4_row(cache, page, h) + (slot - page * cache.page_size);
      const uint32_t c = __ldg(cache.codes[kv] + (row * 8 + j) * groups + g);
      const uint32_t p = __ldg(cache.params[kv] + row * groups + g);
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&p));
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = fmaf(f.x, (float)((c >> (4 * i)) & 15u), f.y);
    }
    put8<T>(static_cast<T*>(out.p[kv]) + token * out.st[kv] + h * out.sh[kv] + 64 * g + 8 * j, x);
  }
}

unsigned kv4_grid(int64_t words) {
  return (unsigned)std::min<int64_t>((words + 255) / 256, (int64_t)sm_count() * 32);
}

}  // namespace

qg_status launch_quantize_kv4(const void* k, int64_t kst, int64_t ksh, const void* v, int64_t vst, int64_t vsh,
                              int dtype, const int64_t* slots, const KV4& cache, int64_t T, cudaStream_t s) {
  const KVIn in = {{k, v}, {kst, vst}, {ksh, vsh}};
  const int wpt = cache.heads * (cache.dim / 8);
  const int64_t words = 2 * T * wpt;
  LaunchCfg lc(kv4_grid(words), 256, 0, s);
  const cudaError_t e =
      dtype == QG_F16 ? cudaLaunchKernelEx(&lc.cfg, quantize_kv4_kernel<__half>, in, slots, cache, words, wpt)
                      : cudaLaunchKernelEx(&lc.cfg, quantize_kv4_kernel<__nv_bfloat16>, in, slots, cache, words, wpt);
  return check_cuda(e, "quantize_kv4 launch");
}

qg_status launch_dequantize_kv4(const KV4& cache, const int64_t* slots, void* k, int64_t kst, int64_t ksh, void* v,
                                int64_t vst, int64_t vsh, int dtype, int64_t T, cudaStream_t s) {
  const KVOut out = {{k, v}, {kst, vst}, {ksh, vsh}};
  const int wpt = cache.heads * (cache.dim / 8);
  const int64_t words = 2 * T * wpt;
  LaunchCfg lc(kv4_grid(words), 256, 0, s);
  const cudaError_t e =
      dtype == QG_F32   ? cudaLaunchKernelEx(&lc.cfg, dequantize_kv4_kernel<float>, out, slots, cache, words, wpt)
      : dtype == QG_F16 ? cudaLaunchKernelEx(&lc.cfg, dequantize_kv4_kernel<__half>, out, slots, cache, words, wpt)
                        : cudaLaunchKernelEx(&lc.cfg, dequantize_kv4_kernel<__nv_bfloat16>, out, slots, cache, words,
                                             wpt);
  return check_cuda(e, "dequantize_kv4 launch");
}

}  // namespace qg
