// qg_norm.cu -- RMS norm with the residual's addition and int8 codes per row
// (the operand of qg_gemm_w8a8), and the reader of int8 rows.
//
// For a row h = x + residual (rounded to the input type) and p = h * w:
//   y = r p with r = 1 / sqrt(mean(h^2) + eps), quantized symmetrically:
//   q = rint(127 y / max|y|) = rint(127 p / max|p|)   (r is common to the row)
//   x_scale = max|y| / 127   = r max|p| / 127
// so a code needs the row's largest |p| only and the norm's factor goes into
// the scale: both reductions (max|p|, sum h^2) come from ONE pass over the
// row, which then stays in registers while its codes are written.  A product
// of two fp16 or bf16 values is exact in binary32, so the codes are bit-exact
// IEEE operations, whatever the order of the sum of squares.
//
// Memory-bound: 7 bytes per element with a residual (x, residual in; h and
// the code out), 3 without; the reader 3 (fp16, bf16) or 5 (fp32).
// 8192 x 4096 with a residual: 37.8 us (6.2 TB/s), reader 17.0 us (5.9 TB/s);
// 1 x 4096: 2.3 and 1.1 us in a row of launches.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cfloat>

#include "qg_device.cuh"
#include "qg_internal.h"

namespace qg {

namespace {

template <typename T>
__device__ __forceinline__ float2 pair_f32(uint32_t v);
template <>
__device__ __forceinline__ float2 pair_f32<__half>(uint32_t v) {
  return __half22float2(*reinterpret_cast<__half2*>(&v));
}
template <>
__device__ __forceinline__ float2 pair_f32<__nv_bfloat16>(uint32_t v) {
  return __bfloat1622float2(*reinterpret_cast<__nv_bfloat162*>(&v));
}

template <typename T>
__device__ __forceinline__ uint32_t pair_bits(float a, float b);
template <>
__device__ __forceinline__ uint32_t pair_bits<__half>(float a, float b) {
  __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<uint32_t*>(&h);
}
template <>
__device__ __forceinline__ uint32_t pair_bits<__nv_bfloat16>(float a, float b) {
  __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<uint32_t*>(&h);
}

// max that returns NaN when either operand is one
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

template <typename T>
__device__ __forceinline__ uint4 add8(uint4 a, uint4 b) {
  uint4 o;
  const uint32_t *pa = &a.x, *pb = &b.x;
  uint32_t* po = &o.x;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 u = pair_f32<T>(pa[i]), v = pair_f32<T>(pb[i]);
    po[i] = pair_bits<T>(__fadd_rn(u.x, v.x), __fadd_rn(u.y, v.y));
  }
  return o;
}

// max |h w| and sum h^2 over 8 elements
template <typename T>
__device__ __forceinline__ void reduce8(uint4 h, uint4 w, float& top, float& ss) {
  const uint32_t *ph = &h.x, *pw = &w.x;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 u = pair_f32<T>(ph[i]), v = pair_f32<T>(pw[i]);
    top = max_nan(top, max_nan(fabsf(__fmul_rn(u.x, v.x)), fabsf(__fmul_rn(u.y, v.y))));
    ss = fmaf(u.x, u.x, fmaf(u.y, u.y, ss));
  }
}

__device__ __forceinline__ int code1(float p, float inv) {
  return max(-127, min(127, __float2int_rn(__fmul_rn(p, inv))));
}

template <typename T>
__device__ __forceinline__ uint2 codes8(uint4 h, uint4 w, float inv) {
  const uint32_t *ph = &h.x, *pw = &w.x;
  uint32_t b[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 u = pair_f32<T>(ph[i]), v = pair_f32<T>(pw[i]);
    const uint32_t lo = (uint32_t)code1(__fmul_rn(u.x, v.x), inv), hi = (uint32_t)code1(__fmul_rn(u.y, v.y), inv);
    b[i] = __byte_perm(lo, hi, 0x0040);  // bytes (lo, hi) in the low half
  }
  return make_uint2(__byte_perm(b[0], b[1], 0x5410), __byte_perm(b[2], b[3], 0x5410));
}

// THREADS threads per row, ROWS rows per block, VEC vectors of 8 elements per
// thread in registers (K <= 8 * VEC * THREADS); VEC = 0: the second pass reads
// h again, from residual_out (or x, without a residual).  residual_out may be
// the residual or x itself: a thread reads its elements before it writes them.
template <typename T, int THREADS, int ROWS, int VEC>
__global__ void __launch_bounds__(THREADS* ROWS)
    rmsnorm_quantize_kernel(const T* x, int64_t ldx, const T* residual, int64_t ldr, const T* __restrict__ weight,
                            float eps, int8_t* __restrict__ xq, int64_t ldq, float* __restrict__ xs, T* res_out,
                            int64_t ldo, int M, int K) {
  constexpr int WARPS = THREADS / 32;
  __shared__ float red_top[ROWS][WARPS], red_ss[ROWS][WARPS];
  pdl_trigger();
  pdl_wait();
  const int r = threadIdx.x / THREADS, t = threadIdx.x % THREADS;
  const int m = blockIdx.x * ROWS + r;
  const bool active = m < M;
  const int64_t row = active ? m : 0;
  const T* xr = x + row * ldx;
  const T* rr = residual ? residual + row * ldr : nullptr;
  T* orow = residual ? res_out + row * ldo : nullptr;
  const uint4* xv = reinterpret_cast<const uint4*>(xr);
  const uint4* rv = reinterpret_cast<const uint4*>(rr);
  const uint4* wv = reinterpret_cast<const uint4*>(weight);
  const int nvec = active ? K / 8 : 0;

  float top = 0.0f, ss = 0.0f;
  uint4 h[VEC > 0 ? VEC : 1];
  if constexpr (VEC > 0) {
    uint4 b[VEC];
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
      const int i = t + j * THREADS;
      h[j] = i < nvec ? xv[i] : make_uint4(0u, 0u, 0u, 0u);
    }
    if (rr) {
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        const int i = t + j * THREADS;
        b[j] = i < nvec ? rv[i] : make_uint4(0u, 0u, 0u, 0u);
      }
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        const int i = t + j * THREADS;
        h[j] = add8<T>(h[j], b[j]);
        if (i < nvec) reinterpret_cast<uint4*>(orow)[i] = h[j];
      }
    }
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
      const int i = t + j * THREADS;
      if (i < nvec) reduce8<T>(h[j], __ldg(wv + i), top, ss);
    }
  } else {
    for (int i = t; i < nvec; i += THREADS) {
      uint4 v = xv[i];
      if (rr) {
        v = add8<T>(v, rv[i]);
        reinterpret_cast<uint4*>(orow)[i] = v;
      }
      reduce8<T>(v, __ldg(wv + i), top, ss);
    }
  }
  // the last K % 8 elements, one per thread (THREADS >= 32 > 7)
  const bool tail = t < K % 8;
  const int kt = K / 8 * 8 + t % 8;
  float tail_p = 0.0f;
  if (active && tail) {
    float v = (float)xr[kt];
    if (rr) {
      const T s = (T)__fadd_rn(v, (float)rr[kt]);
      orow[kt] = s;
      v = (float)s;
    }
    tail_p = __fmul_rn(v, (float)weight[kt]);
    top = max_nan(top, fabsf(tail_p));
    ss = fmaf(v, v, ss);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, o));
    ss += __shfl_xor_sync(0xffffffffu, ss, o);
  }
  if constexpr (WARPS > 1) {
    if ((t & 31) == 0) {
      red_top[r][t / 32] = top;
      red_ss[r][t / 32] = ss;
    }
    __syncthreads();
    top = red_top[r][0];
    ss = red_ss[r][0];
#pragma unroll
    for (int w = 1; w < WARPS; ++w) {
      top = max_nan(top, red_top[r][w]);
      ss += red_ss[r][w];
    }
  }
  if (!active) return;
  const bool finite = top <= FLT_MAX && ss <= FLT_MAX;  // false for NaN
  const float a = fmaxf(top, 1e-30f);
  const float inv = finite ? __fdiv_rn(127.0f, a) : 0.0f;  // p * 0: 0 or NaN, both give the code 0

  int8_t* qrow = xq + row * ldq;
  uint2* qv = reinterpret_cast<uint2*>(qrow);
  if constexpr (VEC > 0) {
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
      const int i = t + j * THREADS;
      if (i < nvec) qv[i] = codes8<T>(h[j], __ldg(wv + i), inv);
    }
  } else {
    const uint4* hv = rr ? reinterpret_cast<const uint4*>(orow) : xv;
    for (int i = t; i < nvec; i += THREADS) qv[i] = codes8<T>(hv[i], __ldg(wv + i), inv);
  }
  if (tail) qrow[kt] = (int8_t)code1(tail_p, inv);
  if (t == 0) {
    const float norm = __fdiv_rn(1.0f, __fsqrt_rn(__fadd_rn(__fdiv_rn(ss, (float)K), eps)));
    xs[m] = finite ? __fmul_rn(__fdiv_rn(a, 127.0f), norm) : __int_as_float(0x7fffffff);
  }
}

template <typename T>
cudaError_t launch_norm(const void* x, int64_t ldx, const void* residual, int64_t ldr, const void* weight, float eps,
                        int8_t* xq, int64_t ldq, float* xs, void* res_out, int64_t ldo, int M, int K,
                        cudaStream_t s) {
  auto go = [&](auto kernel, int threads, int rows) {
    LaunchCfg lc((unsigned)(((int64_t)M + rows - 1) / rows), (unsigned)(threads * rows), 0, s);
    return cudaLaunchKernelEx(&lc.cfg, kernel, static_cast<const T*>(x), ldx, static_cast<const T*>(residual), ldr,
                              static_cast<const T*>(weight), eps, xq, ldq, xs, static_cast<T*>(res_out), ldo, M, K);
  };
  // The row stays in registers up to 8 x 4 x 512 elements.  Few threads with much in flight each carry many rows, more
  // threads shorten the few (us with a residual, chosen / the other):
  //   K <= 1024        1 x 1024: 1.7 / 2.4; 32768 x 1024: 41.9 / 37.2; 65536 x 512, 32 threads a row: 41.5 / 49.8 (64)
  //   K <= 4096        333 x 4096: 3.8 / 4.9 (256 threads); 8192 x 4096: 37.8 / 53.6 (512), 45.5 (two rows of 128 a block)
  //   K <= 16384       1 x 10007: 3.7 / 4.1 (256 threads); 333 x 10007: 6.1 / 8.1 (512)
  const int sms = sm_count();
  if (K <= 1024) {
    if (M <= 4 * sms) return go(rmsnorm_quantize_kernel<T, 128, 1, 1>, 128, 1);
    if (K <= 512) return go(rmsnorm_quantize_kernel<T, 32, 4, 4>, 32, 4);
    return go(rmsnorm_quantize_kernel<T, 64, 2, 2>, 64, 2);
  }
  if (K <= 2048) return go(rmsnorm_quantize_kernel<T, 128, 1, 2>, 128, 1);
  if (K <= 4096 && M > 4 * sms) return go(rmsnorm_quantize_kernel<T, 256, 1, 2>, 256, 1);
  if (K <= 8192) return go(rmsnorm_quantize_kernel<T, 512, 1, 2>, 512, 1);
  if (K <= 16384 && M > sms) return go(rmsnorm_quantize_kernel<T, 256, 1, 8>, 256, 1);
  if (K <= 16384) return go(rmsnorm_quantize_kernel<T, 512, 1, 4>, 512, 1);
  return go(rmsnorm_quantize_kernel<T, 512, 1, 0>, 512, 1);
}

template <typename T>
__device__ __forceinline__ void store8(T* y, const float (&v)[8]);
template <>
__device__ __forceinline__ void store8<float>(float* y, const float (&v)[8]) {
  reinterpret_cast<float4*>(y)[0] = make_float4(v[0], v[1], v[2], v[3]);
  reinterpret_cast<float4*>(y)[1] = make_float4(v[4], v[5], v[6], v[7]);
}
template <>
__device__ __forceinline__ void store8<__half>(__half* y, const float (&v)[8]) {
  *reinterpret_cast<uint4*>(y) = make_uint4(pair_bits<__half>(v[0], v[1]), pair_bits<__half>(v[2], v[3]),
                                            pair_bits<__half>(v[4], v[5]), pair_bits<__half>(v[6], v[7]));
}
template <>
__device__ __forceinline__ void store8<__nv_bfloat16>(__nv_bfloat16* y, const float (&v)[8]) {
  *reinterpret_cast<uint4*>(y) =
      make_uint4(pair_bits<__nv_bfloat16>(v[0], v[1]), pair_bits<__nv_bfloat16>(v[2], v[3]),
                 pair_bits<__nv_bfloat16>(v[4], v[5]), pair_bits<__nv_bfloat16>(v[6], v[7]));
}

template <typename T>
__device__ __forceinline__ void read8(uint2 c, float s, T* y) {
  float v[8];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    v[k] = __fmul_rn((float)(int8_t)(c.x >> (8 * k)), s);
    v[4 + k] = __fmul_rn((float)(int8_t)(c.y >> (8 * k)), s);
  }
  store8<T>(y, v);
}

// Block of 128 threads, threadIdx.x along a row, 8 codes a thread and load, VEC loads in flight: along the row, or
// (BY_ROWS, short rows) of VEC rows.
template <typename T, int VEC, bool BY_ROWS>
__global__ void __launch_bounds__(128) dequantize_rowwise_kernel(const int8_t* __restrict__ xq, int64_t ldq,
                                                                 const float* __restrict__ xs, T* __restrict__ y,
                                                                 int64_t ldy, int M, int K) {
  pdl_trigger();
  pdl_wait();
  const int nvec = K / 8, t = threadIdx.x, kt = nvec * 8 + t % 8;
  const bool tail = t < K % 8;
  if constexpr (BY_ROWS) {
    const int across = blockDim.x, down = blockDim.y;  // down: rows at a time
    const int64_t row0 = (int64_t)blockIdx.x * (VEC * down) + threadIdx.y;
    float s[VEC];
#pragma unroll
    for (int j = 0; j < VEC; ++j) s[j] = row0 + j * down < M ? __ldg(xs + row0 + j * down) : 0.0f;
#pragma unroll 1
    for (int i = t; i < nvec; i += across) {
      uint2 c[VEC];
#pragma unroll
      for (int j = 0; j < VEC; ++j)
        if (row0 + j * down < M) c[j] = __ldg(reinterpret_cast<const uint2*>(xq + (row0 + j * down) * ldq) + i);
#pragma unroll
      for (int j = 0; j < VEC; ++j)
        if (row0 + j * down < M) read8<T>(c[j], s[j], y + (row0 + j * down) * ldy + 8 * i);
    }
    if (tail)
      for (int j = 0; j < VEC; ++j)
        if (row0 + j * down < M) y[(row0 + j * down) * ldy + kt] = (T)__fmul_rn((float)xq[(row0 + j * down) * ldq + kt], s[j]);
  } else {
    const int first = blockIdx.y * (128 * VEC) + t;
    for (int m = blockIdx.x; m < M; m += gridDim.x) {
      const int8_t* q = xq + (int64_t)m * ldq;
      T* out = y + (int64_t)m * ldy;
      const float s = __ldg(xs + m);
#pragma unroll 1
      for (int64_t base = first; base < nvec; base += (int64_t)gridDim.y * (128 * VEC)) {
        uint2 c[VEC];
#pragma unroll
        for (int j = 0; j < VEC; ++j)
          if (base + 128 * j < nvec) c[j] = __ldg(reinterpret_cast<const uint2*>(q) + base + 128 * j);
#pragma unroll
        for (int j = 0; j < VEC; ++j)
          if (base + 128 * j < nvec) read8<T>(c[j], s, out + 8 * (base + 128 * j));
      }
      if (blockIdx.y == 0 && tail) out[kt] = (T)__fmul_rn((float)q[kt], s);
    }
  }
}

template <typename T>
cudaError_t launch_dequant(const int8_t* xq, int64_t ldq, const float* xs, void* y, int64_t ldy, int M, int K,
                           cudaStream_t s) {
  const auto go = [&](auto kernel, LaunchCfg& lc) {
    return cudaLaunchKernelEx(&lc.cfg, kernel, xq, ldq, xs, static_cast<T*>(y), ldy, M, K);
  };
  const int nvec = K / 8;
  // few elements: one load a thread (1 x 4096: 1.1 us, four loads 1.5; 8192 x 4096: 34 and 17)
  const int vec = (int64_t)M * nvec <= (int64_t)sm_count() * 512 ? 1 : 4;
  if (K <= 2048) {  // a block of 128 threads a row would idle or load once (us by rows and not: 32768 x 1024 17, 34)
    int across = 8;
    while (across < std::min(nvec, 128)) across *= 2;
    const int down = 128 / across;
    LaunchCfg lc((unsigned)(((int64_t)M + vec * down - 1) / (vec * down)), (unsigned)across, 0, s);
    lc.cfg.blockDim.y = (unsigned)down;
    return vec == 1 ? go(dequantize_rowwise_kernel<T, 1, true>, lc) : go(dequantize_rowwise_kernel<T, 4, true>, lc);
  }
  LaunchCfg lc((unsigned)M, 128, 0, s);
  lc.cfg.gridDim.y = (unsigned)std::min(std::max(1, (nvec + 128 * vec - 1) / (128 * vec)), 65535);
  return vec == 1 ? go(dequantize_rowwise_kernel<T, 1, false>, lc) : go(dequantize_rowwise_kernel<T, 4, false>, lc);
}

}  // namespace

qg_status launch_rmsnorm_quantize(const void* x, int64_t ldx, const void* residual, int64_t ldr, const void* weight,
                                  int dtype, float eps, int8_t* xq, int64_t ldq, float* xs, void* res_out,
                                  int64_t ldo, int64_t M, int64_t K, cudaStream_t s) {
  const cudaError_t e =
      dtype == QG_F16
          ? launch_norm<__half>(x, ldx, residual, ldr, weight, eps, xq, ldq, xs, res_out, ldo, (int)M, (int)K, s)
          : launch_norm<__nv_bfloat16>(x, ldx, residual, ldr, weight, eps, xq, ldq, xs, res_out, ldo, (int)M,
                                       (int)K, s);
  return check_cuda(e, "rmsnorm_quantize launch");
}

qg_status launch_dequantize_rowwise(const int8_t* xq, int64_t ldq, const float* xs, void* y, int dtype, int64_t ldy,
                                    int64_t M, int64_t K, cudaStream_t s) {
  const cudaError_t e = dtype == QG_F32   ? launch_dequant<float>(xq, ldq, xs, y, ldy, (int)M, (int)K, s)
                        : dtype == QG_F16 ? launch_dequant<__half>(xq, ldq, xs, y, ldy, (int)M, (int)K, s)
                                          : launch_dequant<__nv_bfloat16>(xq, ldq, xs, y, ldy, (int)M, (int)K, s);
  return check_cuda(e, "dequantize_rowwise launch");
}

}  // namespace qg
