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
// Both kernels move 2 + 9/16 bytes per value (a value, its code, 1/64 of its
// group's params), which leaves the issue slots 14 instructions a value at
// HBM's rate.  The writer has 20 and uses 74 % of the slots while it runs; so: no
// conversion instructions (codes go through the mantissa of
// 2^23), minima and maxima in pairs, no division in the common path.  One thread
// owns the 8 channels j of every group of a token's head: one 16-byte access of
// the 16-bit side per group, whose 8 lanes are neighbours, and the group's words
// with one access of the codes, for keys and values of one or more tokens.
//
// 8191 tokens x 8 heads of 128: written in 13.4 us (3.2 TB/s), read in 9.0 (4.8
// TB/s); 32768 x 16 heads of 64 read in 32.3 (5.3 TB/s).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <type_traits>

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
  static __device__ __forceinline__ float2 f32(uint32_t v) { return __half22float2(*reinterpret_cast<V*>(&v)); }
  static __device__ __forceinline__ V round(float a, float b) { return __floats2half2_rn(a, b); }
};
template <>
struct Pair<__nv_bfloat16> {
  using V = __nv_bfloat162;
  static __device__ __forceinline__ float2 f32(uint32_t v) { return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xFFFF0000u)); }
  static __device__ __forceinline__ V round(float a, float b) { return __floats2bfloat162_rn(a, b); }
};

// Minimum of each half of two pairs; NaN where either is one.
template <typename T>
__device__ __forceinline__ uint32_t min2_nan(uint32_t a, uint32_t b) {
  uint32_t d;
  if constexpr (std::is_same<T, __half>::value)
    asm("min.NaN.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  else
    asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

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

// a / 15, correctly rounded: quotient, exact remainder, correction with the rounded reciprocal (Markstein 1990).
// For the tiny a where the remainder would not be exact the result is below the scale's floor.
__device__ __forceinline__ float by_15(float a) {
  const float r = 1.0f / 15.0f, q = a * r;
  return fmaf(fmaf(-15.0f, q, a), r, q);
}

struct KVIn {
  const void* p[2];
  int64_t st[2], sh[2];  // token and head strides (elements)
};

// Codes of 8 values against scale s and offset o, both of the group that holds
// them (so no quotient is below -0.01 or above 15.05: a scale and an offset are
// rounded by less).  The quotient is first taken with an approximate 1/s, off by
// a few 2^-23 of 15; rounding then differs from the division's only next to a
// half-integer, where the 8 are done again with the division.  Adding 1.5 2^23
// rounds half to even and leaves the code in the low bits, so a word is a sum of
// shifted bit patterns less their constant part.
__device__ __forceinline__ uint32_t codes8(const float (&x)[8], float s, float o) {
  constexpr float kMagic = 12582912.0f;  // bits 0x4B400000
  float inv;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(s));
  uint32_t w = 0;
  float far = 0.0f;
#pragma unroll
  for (int i = 7; i >= 0; --i) {
    const float d = __fsub_rn(x[i], o), y = fmaf(d, inv, kMagic);
    far = fmaxf(far, fabsf(fmaf(d, inv, -__fsub_rn(y, kMagic))));
    w = w * 16u + __float_as_uint(y);
  }
  w -= 0x4B400000u * 0x11111111u;
  if (far > 0.4999f) {
    w = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float t = __fdiv_rn(__fsub_rn(x[i], o), s);
      w |= (uint32_t)rintf(fminf(fmaxf(t, 0.0f), 15.0f)) << (4 * i);
    }
  }
  return w;
}

constexpr int kThreads = 128;

// One thread's place: channels 8 j .. of every group of a head, of TOK tokens from `token` on.
struct Place {
  int token, h, j;
};
__device__ __forceinline__ Place place_of(uint32_t u, uint32_t heads, int tok) {
  const uint32_t hu = u >> 3, t = hu / heads;
  return {(int)t * tok, (int)(hu - t * heads), (int)(u & 7)};
}

// Row of a slot in the cache's arrays; -1 for one that is not written or read.
__device__ __forceinline__ int64_t row_of(const KV4& cache, int64_t slot, int64_t limit, int h) {
  if (slot < 0) return -1;
  if (slot >= limit) {
    report_slot();
    return -1;
  }
  const uint32_t page = slot < ((int64_t)1 << 35) ? kv4_page(cache, (uint32_t)(slot >> 4)) : (uint32_t)(slot / cache.page_size);
  const uint32_t in = (uint32_t)slot - page * (uint32_t)cache.page_size;
  return (int64_t)((uint64_t)page * ((uint32_t)cache.heads * (uint32_t)cache.page_size)) +
         ((uint32_t)h * (uint32_t)cache.page_size + in);
}

template <int G>
__device__ __forceinline__ void put_words(uint32_t* p, const uint32_t (&w)[G]) {
  if constexpr (G == 2) *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
  else *p = w[0];
}
template <int G>
__device__ __forceinline__ void get_words(const uint32_t* p, uint32_t (&w)[G]) {
  if constexpr (G == 2) {
    const uint2 v = __ldg(reinterpret_cast<const uint2*>(p));
    w[0] = v.x, w[1] = v.y;
  } else {
    w[0] = __ldg(p);
  }
}

template <typename T, int G, int TOK>
__global__ void __launch_bounds__(kThreads)
    quantize_kv4_kernel(const __grid_constant__ KVIn in, const int64_t* __restrict__ slots,
                        const __grid_constant__ KV4 cache, int tokens, uint32_t units) {
  pdl_trigger();
  pdl_wait();
  const uint32_t u = blockIdx.x * kThreads + threadIdx.x;
  if (u >= units) return;  // units is a multiple of 8: a group's 8 lanes stay together
  const Place at = place_of(u, cache.heads, TOK);
  const int64_t limit = cache.pages * cache.page_size;
  uint4 raw[TOK][2][G];
  int64_t slot[TOK];
#pragma unroll
  for (int i = 0; i < TOK; ++i) slot[i] = at.token + i < tokens ? __ldg(slots + at.token + i) : -1;
#pragma unroll
  for (int kv = 0; kv < 2; ++kv) {
    const T* src = static_cast<const T*>(in.p[kv]) + at.token * in.st[kv] + at.h * in.sh[kv] + 8 * at.j;
#pragma unroll
    for (int i = 0; i < TOK; ++i) {
      const uint4* p = reinterpret_cast<const uint4*>(src + i * in.st[kv]);
#pragma unroll
      for (int g = 0; g < G; ++g) raw[i][kv][g] = at.token + i < tokens ? __ldg(p + 8 * g) : make_uint4(0u, 0u, 0u, 0u);
    }
  }
  const uint32_t mask = 0xFFu << (threadIdx.x & 24);
#pragma unroll
  for (int i = 0; i < TOK; ++i) {
    const int64_t row = row_of(cache, slot[i], limit, at.h);
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
      uint32_t w[G], so[G];
#pragma unroll
      for (int g = 0; g < G; ++g) {
        const uint32_t* rw = &raw[i][kv][g].x;
        // the pairs' minima, and the maxima as minima of the negated values; then over the group's lanes together
        const uint32_t lo = min2_nan<T>(min2_nan<T>(rw[0], rw[1]), min2_nan<T>(rw[2], rw[3]));
        constexpr uint32_t kSign = 0x80008000u;
        const uint32_t hi =
            min2_nan<T>(min2_nan<T>(rw[0] ^ kSign, rw[1] ^ kSign), min2_nan<T>(rw[2] ^ kSign, rw[3] ^ kSign));
        uint32_t both = min2_nan<T>(__byte_perm(lo, hi, 0x5410), __byte_perm(lo, hi, 0x7632));  // (lo, -hi)
#pragma unroll
        for (int d = 4; d > 0; d >>= 1) both = min2_nan<T>(both, __shfl_xor_sync(mask, both, d));
        const float2 lh = Pair<T>::f32(both);
        const float low = min_nan(max_nan(lh.x, -65504.0f), 65504.0f);
        const float high = min_nan(max_nan(-lh.y, -65504.0f), 65504.0f);
        const __half2 h = __floats2half2_rn(max_nan(by_15(__fsub_rn(high, low)), 1e-5f), low);
        so[g] = *reinterpret_cast<const uint32_t*>(&h);
        const float2 f = __half22float2(h);
        float x[8];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float2 v = Pair<T>::f32(rw[k]);
          x[2 * k] = v.x;
          x[2 * k + 1] = v.y;
        }
        const bool inside = lh.x >= -65504.0f && -lh.y <= 65504.0f;  // false for a NaN
        if (!inside) {
#pragma unroll
          for (int k = 0; k < 8; ++k) x[k] = fminf(fmaxf(x[k], -65504.0f), 65504.0f);
        }
        w[g] = codes8(x, f.x, f.y);
        if (!inside && f.x != f.x) w[g] = 0u, so[g] = 0x7FFF7FFFu;
      }
      if (row >= 0) {  // the same for the group's 8 lanes
        put_words<G>(cache.codes[kv] + (row * 8 + at.j) * G, w);
        if (at.j == 0) put_words<G>(cache.params[kv] + row * G, so);
      }
    }
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

template <typename T, int G, int TOK>
__global__ void __launch_bounds__(kThreads)
    dequantize_kv4_kernel(const __grid_constant__ KVOut out, const int64_t* __restrict__ slots,
                          const __grid_constant__ KV4 cache, int tokens, uint32_t units) {
  pdl_trigger();
  pdl_wait();
  const uint32_t u = blockIdx.x * kThreads + threadIdx.x;
  if (u >= units) return;
  const Place at = place_of(u, cache.heads, TOK);
  const int64_t limit = cache.pages * cache.page_size;
  int64_t slot[TOK];
  uint32_t c[TOK][2][G], p[TOK][2][G];
#pragma unroll
  for (int i = 0; i < TOK; ++i) slot[i] = at.token + i < tokens ? __ldg(slots + at.token + i) : -1;
#pragma unroll
  for (int i = 0; i < TOK; ++i) {
    const int64_t row = row_of(cache, slot[i], limit, at.h);
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
#pragma unroll
      for (int g = 0; g < G; ++g) c[i][kv][g] = p[i][kv][g] = 0u;  // scale and offset 0
      if (row >= 0) {
        get_words<G>(cache.codes[kv] + (row * 8 + at.j) * G, c[i][kv]);
        get_words<G>(cache.params[kv] + row * G, p[i][kv]);
      }
    }
  }
#pragma unroll
  for (int kv = 0; kv < 2; ++kv) {
    T* dst = static_cast<T*>(out.p[kv]) + at.token * out.st[kv] + at.h * out.sh[kv] + 8 * at.j;
#pragma unroll
    for (int i = 0; i < TOK; ++i) {
      if (at.token + i >= tokens) break;
#pragma unroll
      for (int g = 0; g < G; ++g) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&p[i][kv][g]));
        float x[8];
        // nibble k of a half word under the mantissa of 2^23 is 2^23 + code 16^k; the scale takes the 16^-k (exact)
        float sk = f.x;
#pragma unroll
        for (int k = 0; k < 4; ++k, sk *= 0.0625f) {
          const uint32_t nibble = 15u << (4 * k), w = c[i][kv][g];
          x[k] = fmaf(sk, __uint_as_float((w & nibble) | 0x4B000000u) - 8388608.0f, f.y);
          x[4 + k] = fmaf(sk, __uint_as_float((w >> 16 & nibble) | 0x4B000000u) - 8388608.0f, f.y);
        }
        put8<T>(dst + i * out.st[kv] + 64 * g, x);
      }
    }
  }
}

// Tokens a thread once that still gives every SM eight blocks of threads; else one (latency).  The writer is a
// chain of load, reduction and store whose instructions fill 74 % of the issue slots, best with 16 channels a thread and many threads (8191 x 8 heads of 128: 13.4 us, two
// tokens a thread 14.4); the reader needs loads in flight, 32 channels (32768 x 16 heads of 64: 32.3 us with four tokens, 37.7 with two, 38.6 with one).
template <int G, bool WRITES>
constexpr int kTokOf = (WRITES ? 2 : 4) / G;
template <int G, bool WRITES>
bool several(int64_t T, int64_t heads) {
  constexpr int kTok = kTokOf<G, WRITES>;
  return kTok > 1 && (T + kTok - 1) / kTok * 8 * heads >= (int64_t)sm_count() * 1024;
}

template <template <typename, int, int> class K, typename T, bool WRITES, class F>
qg_status pick(int dim, int64_t tokens, int64_t heads, F&& go) {
  if (dim == 64) {
    constexpr int kTok = kTokOf<1, WRITES>;
    return several<1, WRITES>(tokens, heads) ? go(K<T, 1, kTok>::fn, kTok) : go(K<T, 1, 1>::fn, 1);
  }
  constexpr int kTok = kTokOf<2, WRITES>;
  return several<2, WRITES>(tokens, heads) ? go(K<T, 2, kTok>::fn, kTok) : go(K<T, 2, 1>::fn, 1);
}
template <typename T, int G, int TOK>
struct Writer {
  static constexpr auto fn = quantize_kv4_kernel<T, G, TOK>;
};
template <typename T, int G, int TOK>
struct Reader {
  static constexpr auto fn = dequantize_kv4_kernel<T, G, TOK>;
};

}  // namespace

qg_status launch_quantize_kv4(const void* k, int64_t kst, int64_t ksh, const void* v, int64_t vst, int64_t vsh,
                              int dtype, const int64_t* slots, const KV4& cache, int64_t T, cudaStream_t s) {
  const KVIn in = {{k, v}, {kst, vst}, {ksh, vsh}};
  auto go = [&](auto kernel, int tok) {
    const int64_t units = (T + tok - 1) / tok * 8 * cache.heads;
    if (units >= ((int64_t)1 << 31)) return fail(QG_ERR_UNSUPPORTED, "quantize_kv4: %lld tokens", (long long)T);
    LaunchCfg lc((unsigned)((units + kThreads - 1) / kThreads), kThreads, 0, s);
    return check_cuda(cudaLaunchKernelEx(&lc.cfg, kernel, in, slots, cache, (int)T, (uint32_t)units), "quantize_kv4 launch");
  };
  return dtype == QG_F16 ? pick<Writer, __half, true>(cache.dim, T, cache.heads, go)
                         : pick<Writer, __nv_bfloat16, true>(cache.dim, T, cache.heads, go);
}

qg_status launch_dequantize_kv4(const KV4& cache, const int64_t* slots, void* k, int64_t kst, int64_t ksh, void* v,
                                int64_t vst, int64_t vsh, int dtype, int64_t T, cudaStream_t s) {
  const KVOut out = {{k, v}, {kst, vst}, {ksh, vsh}};
  auto go = [&](auto kernel, int tok) {
    const int64_t units = (T + tok - 1) / tok * 8 * cache.heads;
    if (units >= ((int64_t)1 << 31)) return fail(QG_ERR_UNSUPPORTED, "dequantize_kv4: %lld tokens", (long long)T);
    LaunchCfg lc((unsigned)((units + kThreads - 1) / kThreads), kThreads, 0, s);
    return check_cuda(cudaLaunchKernelEx(&lc.cfg, kernel, out, slots, cache, (int)T, (uint32_t)units),
                      "dequantize_kv4 launch");
  };
  return dtype == QG_F32   ? pick<Reader, float, false>(cache.dim, T, cache.heads, go)
         : dtype == QG_F16 ? pick<Reader, __half, false>(cache.dim, T, cache.heads, go)
                           : pick<Reader, __nv_bfloat16, false>(cache.dim, T, cache.heads, go);
}

}  // namespace qg
