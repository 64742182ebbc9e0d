// qg_attn_kv4.cu -- attention over the paged 4-bit cache (layout: qg_kv4.cuh).
//
//   out = sum_j p_j v_j / sum_j p_j,  p_j = exp(scale q k_j - m)
// over the visible keys j of a query, in one pass with the running maximum m
// and sum.  One warp per (query token, query head): a lane holds dim / 32
// channels and every key is one dot product across the warp.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "qg_device.cuh"
#include "qg_internal.h"
#include "qg_kv4.cuh"

namespace qg {

static __device__ unsigned long long g_status_prompt;

unsigned long long read_clear_status_prompt(cudaStream_t s) {
  unsigned long long v = 0, z = 0;
  cudaMemcpyFromSymbolAsync(&v, g_status_prompt, sizeof(v), 0, cudaMemcpyDeviceToHost, s);
  cudaMemcpyToSymbolAsync(g_status_prompt, &z, sizeof(z), 0, cudaMemcpyHostToDevice, s);
  cudaStreamSynchronize(s);
  return v;
}

namespace {

__device__ __forceinline__ void report_bad(uint32_t site) {
  atomicCAS(&g_status_prompt, 0ull,
            (unsigned long long)kDevBadArg | ((unsigned long long)site << 8) | ((unsigned long long)blockIdx.x << 24));
}

template <typename T, int DIM>
__global__ void __launch_bounds__(128) attention_kv4_simple(Attn4 a, int min_rows) {
  constexpr int C = DIM / 32;
  pdl_trigger();
  pdl_wait();
  const int lane = threadIdx.x & 31;
  if (blockIdx.x == 0)
    for (int i = threadIdx.x; i < a.B; i += 128) {
      int f, n, l;
      if (!attn4_sequence(a, i, f, n, l)) report_bad(1);
    }
  const int64_t item = (int64_t)blockIdx.x * 4 + threadIdx.x / 32;
  const int t = (int)(item / a.heads_q), hq = (int)(item % a.heads_q);
  if (t >= a.T) return;
  int b, first, n, len;
  if (a.q_starts) {
    int lo = 0, hi = a.B;  // the last b with q_starts[b] <= t
    while (hi - lo > 1) {
      const int mid = (lo + hi) / 2;
      if (__ldg(a.q_starts + mid) <= t) lo = mid;
      else hi = mid;
    }
    b = lo;
  } else {
    b = t / a.n_uniform;
  }
  attn4_sequence(a, b, first, n, len);
  if (t < first || t >= first + n) return;  // a row of no sequence
  if (n * a.group < min_rows) return;       // the decode kernel's
  const int pos = len - n + (t - first);
  const int end = a.causal ? min(len, pos + 1) : len;
  const int begin = a.window > 0 ? max(0, pos - a.window + 1) : 0;

  const int h = hq / a.group, c0 = lane * C;
  const int j = (c0 / 8) % 8, g = c0 / 64, sh = 4 * (c0 % 8);
  constexpr int G = DIM / 64;
  const T* qp = static_cast<const T*>(a.q) + t * a.q_st + hq * a.q_sh + c0;
  float q[C], o[C];
#pragma unroll
  for (int i = 0; i < C; ++i) {
    q[i] = (float)qp[i] * a.scale;
    o[i] = 0.0f;
  }
  float m = -INFINITY, l = 0.0f;
  for (int k = begin; k < end; ++k) {
    const int page_i = k / a.cache.page_size;
    const int page = __ldg(a.table + (int64_t)b * a.table_ld + page_i);
    if (page < 0 || page >= a.cache.pages) {
      report_bad(2);
      continue;
    }
    const int64_t row = kv4_row(a.cache, page, h) + (k - page_i * a.cache.page_size);
    float x[2][C];
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
      const uint32_t c = __ldg(a.cache.codes[kv] + (row * 8 + j) * G + g) >> sh;
      const uint32_t p = __ldg(a.cache.params[kv] + row * G + g);
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&p));
#pragma unroll
      for (int i = 0; i < C; ++i) x[kv][i] = fmaf(f.x, (float)((c >> (4 * i)) & 15u), f.y);
    }
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < C; ++i) s = fmaf(q[i], x[0][i], s);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
    const float mn = fmaxf(m, s);
    const float safe = mn == -INFINITY ? 0.0f : mn;
    const float corr = __expf(m - safe), p = __expf(s - safe);
    l = l * corr + p;
#pragma unroll
    for (int i = 0; i < C; ++i) o[i] = o[i] * corr + p * x[1][i];
    m = mn;
  }
  T* op = static_cast<T*>(a.out) + t * a.o_st + hq * a.o_sh + c0;
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
#pragma unroll
  for (int i = 0; i < C; ++i) op[i] = (T)(l == 0.0f ? 0.0f : o[i] * inv);
  if (a.lse && lane == 0) a.lse[(int64_t)t * a.heads_q + hq] = l == 0.0f ? -INFINITY : m + logf(l);
}

}  // namespace

// Rows (query tokens x head group) that the decode kernel takes, in tiles of 8;
// 0: none.  Ragged calls give it the sequences of one tile's size or less.
static int decode_tiles(int64_t n, int64_t group, bool ragged) {
  const int64_t rows = ragged ? group : n * group;
  return rows <= 8 ? 1 : rows <= 16 ? 2 : 0;
}

size_t attention_kv4_workspace(int64_t B, int64_t T, int64_t heads_q, int64_t heads, int64_t dim, bool ragged) {
  const int nt = decode_tiles(T / B, heads_q / heads, ragged);
  return nt ? attention_kv4_decode_workspace(dim, nt) : 0;
}

qg_status launch_attention_kv4(const Attn4& a, void* workspace, cudaStream_t s) {
  const int nt = decode_tiles(a.n_uniform, a.group, a.q_starts != nullptr);
  if (nt) {
    const qg_status st = launch_attention_kv4_decode(a, nt, workspace, s);
    if (st != QG_OK || !a.q_starts) return st;
  }
  const int64_t items = (int64_t)a.T * a.heads_q;
  const int min_rows = 8 * nt + 1;
  LaunchCfg lc((unsigned)((items + 3) / 4), 128, 0, s);
  cudaError_t e;
  if (a.dtype == QG_F16)
    e = a.cache.dim == 64 ? cudaLaunchKernelEx(&lc.cfg, attention_kv4_simple<__half, 64>, a, min_rows)
                          : cudaLaunchKernelEx(&lc.cfg, attention_kv4_simple<__half, 128>, a, min_rows);
  else
    e = a.cache.dim == 64 ? cudaLaunchKernelEx(&lc.cfg, attention_kv4_simple<__nv_bfloat16, 64>, a, min_rows)
                          : cudaLaunchKernelEx(&lc.cfg, attention_kv4_simple<__nv_bfloat16, 128>, a, min_rows);
  return check_cuda(e, "attention_kv4 launch");
}

}  // namespace qg
