// qg_attn_kv4_decode.cu -- attention of few query rows over the paged 4-bit
// cache: every (sequence, KV head) whose query tokens times head group make at
// most 16 rows (single-token decode, draft tokens).
//
// Memory-bound in principle: a key and value of 128 channels are 144 bytes, so
// at HBM rate an SM has about 6 cycles for the 256 codes of a token.  What
// decides the time is therefore the instructions per code, and the codes are
// never dequantized one by one:
//   score_j = sum_g [ s_jg (q_g . c_jg) + o_jg sum(q_g) ]
//   out     = sum_j p_j (s_jg c_j + o_jg) = sum_j (p_j s_jg) (c_j - 8) + sum_j p_j (o_jg + 8 s_jg)
// (g: group of 64 channels; s, o: its scale and offset; c: codes).  The products
// run on the codes themselves.  A nibble masked into the low bits of a half is
// the fp16 subnormal c 2^-24 (or, four bits up, 16 c 2^-24), exact on the tensor
// cores: two codes cost one mask, with one shift per four.  Queries are scaled
// by a power of two to fp16 (1/16 of it where they meet a nibble four bits up),
// scale and offset enter per token and group in binary32.  p s is rounded to
// fp16 under a power of two kappa (a shift of the running maximum) that keeps
// the largest near 2^8.  Codes are
// taken from their middle (a second product with the constant -8, cheaper than
// changing the codes) because values have either sign: without it the sum over
// n keys is large against the result and its truncation shows (0.0013 instead
// of 0.0003 relative error at 131071 keys).
//
// mma.m16n8k16 with keys (16 tokens) or channels (16 of V^T) as its rows and up
// to 8 query rows as its columns: the accumulators of q.c and of the output
// have the same columns in the same lanes, so the running maximum needs no
// exchange, and movmatrix turns the probabilities into the second product's
// operand.  (tcgen05 would take the codes through shared or tensor memory:
// more bytes moved per code than this has instructions.)
//
// Every warp is a worker of its own: the chunks of 64 tokens of all sequences
// and heads form one list, split evenly over the warps of one CTA per SM, so
// ragged lengths balance.  A warp streams its share through a ring of
// bulk copies (one per page piece and array) without any block barrier.  A
// (sequence, head) that one warp covers is written at once; the parts of one
// that several cover are joined by a second kernel in list order (no atomics).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "qg_device.cuh"
#include "qg_internal.h"
#include "qg_kv4.cuh"

namespace qg {

static __device__ unsigned long long g_status_attn;

unsigned long long read_clear_status_attn(cudaStream_t s) {
  unsigned long long v = 0, z = 0;
  cudaMemcpyFromSymbolAsync(&v, g_status_attn, sizeof(v), 0, cudaMemcpyDeviceToHost, s);
  cudaMemcpyToSymbolAsync(g_status_attn, &z, sizeof(z), 0, cudaMemcpyHostToDevice, s);
  cudaStreamSynchronize(s);
  return v;
}

namespace {

constexpr int kChunk = 64;   // tokens per ring stage
constexpr int kWarps = 8;    // workers per CTA
constexpr int kStages = 2;
constexpr uint32_t kMinus8 = 0x80088008u, kMinus128 = 0x80808080u;  // fp16x2: -8 2^-24, -128 2^-24

// device status sites
enum : uint32_t { kSiteSequence = 1, kSitePage = 2, kSiteWait = 3 };

__device__ __forceinline__ void report(uint32_t code, uint32_t site) {
  atomicCAS(&g_status_attn, 0ull,
            (unsigned long long)code | ((unsigned long long)site << 8) | ((unsigned long long)blockIdx.x << 24));
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The same with a zero accumulator.
__device__ __forceinline__ void mma16816_zero(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                              uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
}

// max of each signed 16-bit half
__device__ __forceinline__ uint32_t max_halves(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("max.s16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t a) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}

__device__ __forceinline__ uint32_t half2_bits(float lo, float hi) {
  __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&h);
}

__device__ __forceinline__ float2 half2_f32(uint32_t v) {
  return __half22float2(*reinterpret_cast<__half2*>(&v));
}

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst), "l"(src),
      "r"(bytes), "r"(bar)
      : "memory");
}

template <int N>
__device__ __forceinline__ void lds(uint32_t (&r)[N], uint32_t addr) {
  static_assert(N == 1 || N == 2 || N == 4, "");
  if constexpr (N == 1)
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(r[0]) : "r"(addr));
  else if constexpr (N == 2)
    asm volatile("ld.shared.v2.b32 {%0,%1}, [%2];" : "=r"(r[0]), "=r"(r[1]) : "r"(addr));
  else
    asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr));
}

// What a sequence asks of this kernel: its chunks [c0, c0 + chunks) per head.
struct Seq {
  int first, n, len, lo, c0, chunks;
};

template <int NT>
__device__ __forceinline__ Seq sequence(const Attn4& a, int b, bool& ok) {
  Seq s;
  ok = attn4_sequence(a, b, s.first, s.n, s.len);
  // the oldest key that any query sees
  s.lo = a.window > 0 ? max(0, min(s.len, s.len - s.n - a.window + 1)) : 0;
  s.c0 = s.lo / kChunk;
  s.chunks = s.n == 0 || s.n > 8 * NT / a.group ? 0 : max(1, (s.len + kChunk - 1) / kChunk - s.c0);
  return s;
}

// Position in the list of chunks
template <int NT>
struct Cursor {
  int b, h, c;
  Seq s;
  __device__ __forceinline__ void next(const Attn4& a) {
    if (++c < s.chunks) return;
    c = 0;
    if (++h < a.cache.heads) return;
    h = 0;
    bool ok;
    do {
      if (++b >= a.B) return;
      s = sequence<NT>(a, b, ok);
    } while (s.chunks == 0);
  }
};

// Workers share the list evenly: worker w of W has units [U w / W, U (w + 1) / W).
__device__ __forceinline__ int64_t share(int64_t U, int64_t w, int64_t W) { return U * w / W; }
__device__ __forceinline__ int worker_of(int64_t unit, int64_t U, int64_t W) { return (int)(((unit + 1) * W - 1) / U); }

// One worker's part of a (sequence, head): rows of dim sums, then m and l.
__host__ __device__ constexpr int part_floats(int nt, int dim) { return 8 * nt * (dim + 2); }

template <int G, int NT>
__global__ void __launch_bounds__(32 * kWarps, 1)
    attention_kv4_decode(const __grid_constant__ Attn4 a, int32_t* __restrict__ prefix_out, float* __restrict__ parts) {
  constexpr int D = 64 * G;
  constexpr uint32_t kCodes = kChunk * D / 2, kParams = kChunk * G * 4;
  constexpr uint32_t kStage = 2 * (kCodes + kParams);
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ __align__(8) uint64_t bars[kWarps][kStages];
  __shared__ int warp_sums[kWarps];
  int* prefix = reinterpret_cast<int*>(smem + kWarps * kStages * kStage);

  const int tid = threadIdx.x, lane = tid & 31, warp = tid / 32;
  const int q4 = lane & 3, r8 = lane >> 2;
  if (lane == 0) {
#pragma unroll
    for (int i = 0; i < kStages; ++i) mbar_init(smem_u32(&bars[warp][i]), 1);
    fence_mbar_init();
  }
  pdl_trigger();
  pdl_wait();

  // prefix[b]: chunks (times heads) of the sequences before b
  {
    const int per = (a.B + 32 * kWarps - 1) / (32 * kWarps);
    int sum = 0;
    bool ok;
    for (int i = 0; i < per; ++i) {
      const int b = tid * per + i;
      if (b < a.B) {
        sum += sequence<NT>(a, b, ok).chunks * a.cache.heads;
        if (!ok && blockIdx.x == 0) report(kDevBadArg, kSiteSequence);
      }
    }
    int scan = sum;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, scan, d);
      if (lane >= d) scan += v;
    }
    if (lane == 31) warp_sums[warp] = scan;
    __syncthreads();
    int at = scan - sum;
    for (int w = 0; w < warp; ++w) at += warp_sums[w];
    for (int i = 0; i < per; ++i) {
      const int b = tid * per + i;
      if (b < a.B) {
        prefix[b] = at;
        at += sequence<NT>(a, b, ok).chunks * a.cache.heads;
        if (b == a.B - 1) prefix[a.B] = at;
      }
    }
    __syncthreads();
    if (blockIdx.x == 0)
      for (int b = tid; b <= a.B; b += 32 * kWarps) prefix_out[b] = prefix[b];
  }
  const int64_t U = prefix[a.B];
  const int64_t W = min(U, (int64_t)gridDim.x * kWarps);
  const int w = warp * gridDim.x + blockIdx.x;  // neighbours in the list on different SMs
  if (w >= W) return;
  const int u0 = (int)share(U, w, W), u1 = (int)share(U, w + 1, W);

  Cursor<NT> fill;
  {
    int lo = 0, hi = a.B;  // the last b with prefix[b] <= u0 (its chunks are not 0)
    while (hi - lo > 1) {
      const int mid = (lo + hi) / 2;
      if (prefix[mid] <= u0) lo = mid;
      else hi = mid;
    }
    bool ok;
    fill.b = lo;
    fill.s = sequence<NT>(a, lo, ok);
    const int in = u0 - prefix[lo];
    fill.h = in / fill.s.chunks;
    fill.c = in - fill.h * fill.s.chunks;
  }
  Cursor<NT> use = fill;

  // --- the ring -------------------------------------------------------------
  const uint32_t ring = smem_u32(smem) + warp * kStages * kStage;
  const int P = a.cache.page_size;
  const int piece = min(kChunk, P & -P);  // tokens per copy: 16, 32 or 64, never across a page's end
  const int pieces = kChunk / piece;
  // lane (array, piece): 0 key codes, 1 value codes, 2 key params, 3 value params
  const int arr = lane / pieces, pc = lane % pieces;
  const bool copies = arr < 4;
  const uint32_t bytes = arr < 2 ? piece * (D / 2) : piece * (G * 4);
  const uint32_t dst_off = (arr < 2 ? arr * kCodes : 2 * kCodes + (arr - 2) * kParams) + pc * bytes;
  const uint32_t code_lanes = (1u << (2 * pieces)) - 1;

  int page = -1, in_page = 0;  // of the lane's piece of the next chunk to fill; page -1: nothing
  auto look_up = [&]() {
    page = -1;
    const int t = (fill.s.c0 + fill.c) * kChunk + pc * piece;
    if (copies && t < fill.s.len) {
      const int i = t / P;
      in_page = t - i * P;
      page = __ldg(a.table + (int64_t)fill.b * a.table_ld + i);
      if (page < 0 || page >= a.cache.pages) {
        report(kDevBadArg, kSitePage);
        page = -1;
      }
    }
  };
  auto issue = [&](int stage) {  // the whole warp
    const uint32_t have = __ballot_sync(0xffffffffu, page >= 0);
    const uint32_t bar = smem_u32(&bars[warp][stage]);
    if (lane == 0)
      mbar_arrive_expect_tx(bar, __popc(have & code_lanes) * (uint32_t)(piece * (D / 2)) +
                                     __popc(have & ~code_lanes) * (uint32_t)(piece * (G * 4)));
    __syncwarp();
    if (page >= 0) {
      const int64_t row = kv4_row(a.cache, page, fill.h) + in_page;
      const uint32_t* src = arr < 2 ? (arr == 0 ? a.cache.codes[0] : a.cache.codes[1]) + row * (D / 8)
                                    : (arr == 2 ? a.cache.params[0] : a.cache.params[1]) + row * G;
      bulk_load(ring + stage * kStage + dst_off, src, bytes, bar);
    }
  };

  const int units = u1 - u0;
  look_up();
#pragma unroll 1
  for (int i = 0; i < kStages && i < units; ++i) {
    issue(i);
    if (i + 1 < units) {
      fill.next(a);
      look_up();
    }
  }

  // --- the item in hand -------------------------------------------------------
  uint32_t qf[NT][G][2][4];        // queries, the second operand of q . c
  float qs[NT][2][G];              // sums of the group's queries, times 2^-24: columns 2 q4, 2 q4 + 1
  float sigma[NT][2];              // scale log2(e) 2^24 over the queries' power of two
  float m[NT][2], l[NT][2];        // running maximum (before sigma) and sum
  float ob[NT][2][G];              // sum p o
  float o[NT][G][4][4];            // sum p s (c - 8) 2^-24
  int end[NT][2], beg[NT][2];      // visible keys of the columns
  float lift = 0.0f, lifted = 1.0f;  // log2 kappa, kappa: l, ob and o hold p kappa
  bool fresh = true, starts_item = false;
  int min_end = 0, max_beg = 0;    // keys that every row sees

  auto begin_item = [&]() {
    const Seq& s = use.s;
    const int rows = s.n * a.group;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int row = nt * 8 + r8;
      float x[G][2][8];
      float amax = 0.0f;
#pragma unroll
      for (int g = 0; g < G; ++g)
#pragma unroll
        for (int jj = 0; jj < 2; ++jj) {
          uint4 v = make_uint4(0u, 0u, 0u, 0u);
          if (row < rows) {
            const int t = s.first + row / a.group, hq = use.h * a.group + row % a.group;
            const char* p = static_cast<const char*>(a.q) +
                            2 * (t * a.q_st + hq * a.q_sh + 64 * g + 8 * (2 * q4 + jj));
            v = *reinterpret_cast<const uint4*>(p);
          }
          const uint32_t* pv = &v.x;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint32_t b = pv[i];
            const float2 f = a.dtype == QG_F16 ? half2_f32(b)
                                               : make_float2(__uint_as_float(b << 16), __uint_as_float(b & 0xffff0000u));
            x[g][jj][2 * i] = f.x;
            x[g][jj][2 * i + 1] = f.y;
            amax = fmaxf(amax, fmaxf(fabsf(f.x), fabsf(f.y)));
          }
        }
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
      // largest query near 2^8: exact in fp16 down to 2^-22 of it, also after the 1/16
      int e = 8 - ((int)(__float_as_uint(amax) >> 23) - 127);
      e = max(-100, min(100, e));
      const float up = __uint_as_float((uint32_t)(127 + e) << 23);
      const float sg = a.scale * 1.44269504088896f * 16777216.0f * __uint_as_float((uint32_t)(127 - e) << 23);
      float sum[G];
#pragma unroll
      for (int g = 0; g < G; ++g) {
        sum[g] = 0.0f;
#pragma unroll
        for (int jj = 0; jj < 2; ++jj) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            x[g][jj][i] *= up;
            sum[g] += x[g][jj][i];
          }
          qf[nt][g][jj][0] = half2_bits(x[g][jj][0], x[g][jj][4]);
          qf[nt][g][jj][1] = half2_bits(x[g][jj][1] * 0.0625f, x[g][jj][5] * 0.0625f);
          qf[nt][g][jj][2] = half2_bits(x[g][jj][2], x[g][jj][6]);
          qf[nt][g][jj][3] = half2_bits(x[g][jj][3] * 0.0625f, x[g][jj][7] * 0.0625f);
        }
        sum[g] += __shfl_xor_sync(0xffffffffu, sum[g], 1);
        sum[g] += __shfl_xor_sync(0xffffffffu, sum[g], 2);
      }
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int from = 4 * (2 * q4 + c);
        sigma[nt][c] = __shfl_sync(0xffffffffu, sg, from);
#pragma unroll
        for (int g = 0; g < G; ++g) {
          qs[nt][c][g] = __shfl_sync(0xffffffffu, sum[g], from) * 5.9604644775390625e-8f;
          ob[nt][c][g] = 0.0f;
        }
        m[nt][c] = -INFINITY;
        l[nt][c] = 0.0f;
        const int col = nt * 8 + 2 * q4 + c;
        const int pos = s.len - s.n + min(col, rows - 1) / a.group;
        end[nt][c] = a.causal ? min(s.len, pos + 1) : s.len;
        beg[nt][c] = a.window > 0 ? max(0, pos - a.window + 1) : 0;
      }
#pragma unroll
      for (int g = 0; g < G; ++g)
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int k = 0; k < 4; ++k) o[nt][g][i][k] = 0.0f;
    }
    min_end = a.causal ? s.len - s.n + 1 : s.len;
    max_beg = a.window > 0 ? s.len - a.window : 0;
    fresh = true;
    lift = 0.0f;
    starts_item = use.c == 0;
  };

  auto end_item = [&](bool whole) {
    const Seq& s = use.s;
    const int rows = s.n * a.group;
    float* part = parts + (int64_t)(2 * w + (starts_item ? 1 : 0)) * part_floats(NT, D);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) {
          l[nt][c] += __shfl_xor_sync(0xffffffffu, l[nt][c], d);
#pragma unroll
          for (int g = 0; g < G; ++g) ob[nt][c][g] += __shfl_xor_sync(0xffffffffu, ob[nt][c][g], d);
        }
        const int row = nt * 8 + 2 * q4 + c;
        if (row >= rows) continue;
        const float top = m[nt][c] * sigma[nt][c] - lift;  // log2 units; -inf: nothing seen
        const int t = s.first + row / a.group, hq = use.h * a.group + row % a.group;
        const float inv = l[nt][c] == 0.0f ? 0.0f : 1.0f / l[nt][c];
#pragma unroll
        for (int g = 0; g < G; ++g) {
          float v[8];
          // tile i, row r8 and r8 + 8: nibbles (0, 2), (1, 3), (4, 6), (5, 7)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float f = i & 1 ? 1048576.0f : 16777216.0f;
            const int ka = (i >> 1) * 4 + (i & 1);
            v[ka] = fmaf(o[nt][g][i][c], f, ob[nt][c][g]);
            v[ka + 2] = fmaf(o[nt][g][i][2 + c], f, ob[nt][c][g]);
          }
          if (whole) {
            uint32_t b[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float x = l[nt][c] == 0.0f ? 0.0f : v[2 * i] * inv, y = l[nt][c] == 0.0f ? 0.0f : v[2 * i + 1] * inv;
              if (a.dtype == QG_F16) {
                b[i] = half2_bits(x, y);
              } else {
                __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
                b[i] = *reinterpret_cast<uint32_t*>(&h);
              }
            }
            char* p = static_cast<char*>(a.out) + 2 * (t * a.o_st + hq * a.o_sh + 64 * g + 8 * r8);
            *reinterpret_cast<uint4*>(p) = make_uint4(b[0], b[1], b[2], b[3]);
          } else {
            float4* p = reinterpret_cast<float4*>(part + row * D + 64 * g + 8 * r8);
            p[0] = make_float4(v[0], v[1], v[2], v[3]);
            p[1] = make_float4(v[4], v[5], v[6], v[7]);
          }
        }
        if (r8 == 0) {
          if (!whole) {
            part[8 * NT * D + 2 * row] = top;
            part[8 * NT * D + 2 * row + 1] = l[nt][c];
          } else if (a.lse) {
            a.lse[(int64_t)t * a.heads_q + hq] = l[nt][c] == 0.0f ? -INFINITY : (top + log2f(l[nt][c])) * 0.69314718056f;
          }
        }
      }
  };

  begin_item();
  // the token of fragment row r (0..7): pairs (0,1), (3,2), (4,5), (7,6), which spreads the value loads over the banks
  const int kt = r8 ^ ((r8 >> 1) & 1);
  const int vt0 = 2 * q4 + (q4 & 1), vt1 = vt0 ^ 1;  // rows 2 q4 and 2 q4 + 1
  uint32_t phases = 0;

#pragma unroll 1
  for (int i = 0; i < units; ++i) {
    const int stage = i % kStages;
    if (!mbar_wait(smem_u32(&bars[warp][stage]), (phases >> stage) & 1, &g_status_attn, kSiteWait)) {
      // give up: let the other copies in flight land (bounded), then leave
      for (int k = 1; k < kStages && i + k < units; ++k)
        mbar_wait(smem_u32(&bars[warp][(i + k) % kStages]), (phases >> ((i + k) % kStages)) & 1, &g_status_attn, kSiteWait);
      return;
    }
    phases ^= 1u << stage;
    const uint32_t base = ring + stage * kStage;
    const uint32_t kc = base, vc = base + kCodes, kp = base + 2 * kCodes, vp = kp + kParams;
    const int t0 = (use.s.c0 + use.c) * kChunk;
    auto chunk = [&](auto all) {  // all: every row sees every key
      constexpr bool kAll = decltype(all)::value;
      // scores
      float x[NT][4][4];
#pragma unroll
      for (int tile = 0; tile < 4; ++tile) {
        uint32_t kw[2][2 * G], pw[2][G];
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {
          const int tok = tile * 16 + hh * 8 + kt;
          lds(kw[hh], kc + tok * (D / 2) + q4 * (8 * G));
          lds(pw[hh], kp + tok * (G * 4));
        }
        float acc[NT][G][4];
#pragma unroll
        for (int jj = 0; jj < 2; ++jj)
#pragma unroll
          for (int g = 0; g < G; ++g) {
            const uint32_t u = kw[0][jj * G + g], v = kw[1][jj * G + g];
            const uint32_t us = u >> 8, vs = v >> 8;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              if (jj == 0)
                mma16816_zero(acc[nt][g], u & 0x000F000Fu, v & 0x000F000Fu, u & 0x00F000F0u, v & 0x00F000F0u,
                              qf[nt][g][jj][0], qf[nt][g][jj][1]);
              else
                mma16816(acc[nt][g], u & 0x000F000Fu, v & 0x000F000Fu, u & 0x00F000F0u, v & 0x00F000F0u,
                         qf[nt][g][jj][0], qf[nt][g][jj][1]);
              mma16816(acc[nt][g], us & 0x000F000Fu, vs & 0x000F000Fu, us & 0x00F000F0u, vs & 0x00F000F0u,
                       qf[nt][g][jj][2], qf[nt][g][jj][3]);
            }
          }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            float v = 0.0f;
#pragma unroll
            for (int g = 0; g < G; ++g) {
              const float2 so = half2_f32(pw[k >> 1][g]);
              v = g == 0 ? so.y * qs[nt][k & 1][g] : fmaf(so.y, qs[nt][k & 1][g], v);
              v = fmaf(acc[nt][g][k], so.x, v);
            }
            if constexpr (!kAll) {
              const int t = t0 + tile * 16 + (k >> 1) * 8 + kt;
              if (t < beg[nt][k & 1] || t >= end[nt][k & 1]) v = -INFINITY;
            }
            x[nt][tile][k] = v;
          }
      }

      // the values' params; the largest scale among keys that any row sees
      uint32_t vw[4][2][G];
      uint32_t smax = 0;
#pragma unroll
      for (int tile = 0; tile < 4; ++tile)
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {
          const int tok = tile * 16 + hh * 8 + kt;
          lds(vw[tile][hh], vp + tok * (G * 4));
          const bool in = kAll || (t0 + tok >= use.s.lo && t0 + tok < use.s.len);
#pragma unroll
          for (int g = 0; g < G; ++g)
            if (in) smax = max_halves(smax, vw[tile][hh][g]);
        }
      // fp16 bits order like the values (a scale is not negative)
      smax = min(__reduce_max_sync(0xffffffffu, smax & 0x7FFFu), 0x7BFFu);
      const float stop = __half2float(__ushort_as_half((unsigned short)smax));
      float shift = lift;
      if (fresh || stop * lifted > 32768.0f) {  // a first scale, or one that p s kappa would not hold in fp16
        const int e = min(40, 8 - ((int)(__float_as_uint(stop) >> 23) - 127));
        lifted = __uint_as_float((uint32_t)(127 + e) << 23);
        lift = (float)e;
        fresh = false;
      }
      shift = lift - shift;

      // running maximum
      bool moved = shift != 0.0f;
      float corr[NT][2], mneg[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          float t = m[nt][c];
#pragma unroll
          for (int tile = 0; tile < 4; ++tile) t = fmaxf(t, fmaxf(x[nt][tile][c], x[nt][tile][2 + c]));
#pragma unroll
          for (int d = 4; d < 32; d <<= 1) t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, d));
          const float safe = t == -INFINITY ? 0.0f : t;
          corr[nt][c] = ex2(fmaf(m[nt][c] - safe, sigma[nt][c], shift));
          moved |= t != m[nt][c];
          m[nt][c] = t;
          mneg[nt][c] = fmaf(-safe, sigma[nt][c], lift);
        }
      if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            l[nt][c] *= corr[nt][c];
#pragma unroll
            for (int g = 0; g < G; ++g) {
              ob[nt][c][g] *= corr[nt][c];
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                o[nt][g][k][c] *= corr[nt][c];
                o[nt][g][k][2 + c] *= corr[nt][c];
              }
            }
          }
      }

      // probabilities (times kappa) and the second product
#pragma unroll
      for (int tile = 0; tile < 4; ++tile) {
        uint32_t pf[NT][G][2];
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {
          float2 so[G];
#pragma unroll
          for (int g = 0; g < G; ++g) {
            so[g] = half2_f32(vw[tile][hh][g]);
            so[g].y = fmaf(8.0f, so[g].x, so[g].y);
          }
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            float p[2];
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              p[c] = ex2(fmaf(x[nt][tile][2 * hh + c], sigma[nt][c], mneg[nt][c]));
              l[nt][c] += p[c];
            }
#pragma unroll
            for (int g = 0; g < G; ++g) {
              float ps[2];
#pragma unroll
              for (int c = 0; c < 2; ++c) {
                if (kAll || x[nt][tile][2 * hh + c] != -INFINITY) {  // a hidden key's params may be anything
                  ps[c] = p[c] * so[g].x;
                  ob[nt][c][g] = fmaf(p[c], so[g].y, ob[nt][c][g]);
                } else {
                  ps[c] = 0.0f;
                }
              }
              pf[nt][g][hh] = transpose8x8(half2_bits(ps[0], ps[1]));
            }
          }
        }
        uint32_t v0[2][G], v1[2][G];
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {
          lds(v0[hh], vc + (tile * 16 + hh * 8 + vt0) * (D / 2) + r8 * (4 * G));
          lds(v1[hh], vc + (tile * 16 + hh * 8 + vt1) * (D / 2) + r8 * (4 * G));
        }
#pragma unroll
        for (int g = 0; g < G; ++g) {
#pragma unroll
          for (int half = 0; half < 2; ++half) {  // nibbles 0..3, 4..7
            const uint32_t sel = half ? 0x7632u : 0x5410u;
            const uint32_t e = __byte_perm(v0[0][g], v1[0][g], sel), f = __byte_perm(v0[1][g], v1[1][g], sel);
            const uint32_t es = e >> 8, fs = f >> 8;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              mma16816(o[nt][g][2 * half], e & 0x000F000Fu, es & 0x000F000Fu, f & 0x000F000Fu, fs & 0x000F000Fu,
                       pf[nt][g][0], pf[nt][g][1]);
              mma16816(o[nt][g][2 * half], kMinus8, kMinus8, kMinus8, kMinus8, pf[nt][g][0], pf[nt][g][1]);
              mma16816(o[nt][g][2 * half + 1], e & 0x00F000F0u, es & 0x00F000F0u, f & 0x00F000F0u, fs & 0x00F000F0u,
                       pf[nt][g][0], pf[nt][g][1]);
              mma16816(o[nt][g][2 * half + 1], kMinus128, kMinus128, kMinus128, kMinus128, pf[nt][g][0], pf[nt][g][1]);
            }
          }
        }
      }
    };
    if (t0 >= max_beg && t0 + kChunk <= min_end) chunk(std::true_type{});
    else chunk(std::false_type{});

    // refill the stage
    __syncwarp();
    if (i + kStages < units) {
      issue(stage);
      if (i + kStages + 1 < units) {
        fill.next(a);
        look_up();
      }
    }
    // the item's end, or the worker's
    const bool item_done = use.c + 1 == use.s.chunks;
    if (item_done || i + 1 == units) end_item(item_done && starts_item);
    if (i + 1 < units) {
      use.next(a);
      if (item_done) begin_item();
    }
  }
}

// Joins the parts of the (sequence, head)s that several workers share: block
// (row, head, sequence), a warp per part in turn, the sums over warps in order.
template <int D>
__global__ void __launch_bounds__(256)
    attention_kv4_join(const __grid_constant__ Attn4 a, const int32_t* __restrict__ prefix,
                       const float* __restrict__ parts, int workers, int nt) {
  constexpr int V = D / 32;  // values per lane
  __shared__ float sums[8][D];
  __shared__ float ls[8];
  pdl_trigger();
  pdl_wait();
  const int row = blockIdx.x, h = blockIdx.y, b = blockIdx.z;
  const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
  const int i0 = prefix[b], i1 = prefix[b + 1];
  if (i1 == i0) return;
  int first, n, len;
  attn4_sequence(a, b, first, n, len);
  if (row >= n * a.group) return;
  const int64_t U = prefix[a.B], W = min(U, (int64_t)workers);
  const int chunks = (i1 - i0) / a.cache.heads;
  const int64_t u = i0 + (int64_t)h * chunks;
  const int wa = worker_of(u, U, W), wb = worker_of(u + chunks - 1, U, W);
  if (wa == wb) return;
  const int rows = 8 * nt, stride = rows * (D + 2), count = wb - wa + 1;
  auto part = [&](int i) { return parts + (int64_t)(2 * (wa + i) + (i == 0 ? 1 : 0)) * stride; };

  float top = -INFINITY;
  for (int i = lane; i < count; i += 32) top = fmaxf(top, part(i)[rows * D + 2 * row]);
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
  const float safe = top == -INFINITY ? 0.0f : top;
  float acc[V] = {}, l = 0.0f;
#pragma unroll 4
  for (int i = warp; i < count; i += 8) {
    const float* p = part(i);
    const float2 ml = *reinterpret_cast<const float2*>(p + rows * D + 2 * row);
    const float f = ex2(ml.x - safe);
    l += ml.y * f;
    float v[V];
    if constexpr (V == 4)
      *reinterpret_cast<float4*>(v) = *reinterpret_cast<const float4*>(p + row * D + V * lane);
    else
      *reinterpret_cast<float2*>(v) = *reinterpret_cast<const float2*>(p + row * D + V * lane);
#pragma unroll
    for (int k = 0; k < V; ++k) acc[k] = fmaf(v[k], f, acc[k]);
  }
#pragma unroll
  for (int k = 0; k < V; ++k) sums[warp][V * lane + k] = acc[k];
  if (lane == 0) ls[warp] = l;
  __syncthreads();
  float total = 0.0f;
#pragma unroll
  for (int w = 0; w < 8; ++w) total += ls[w];
  const int t = first + row / a.group, hq = h * a.group + row % a.group;
  if (threadIdx.x < D) {
    float v = 0.0f;
#pragma unroll
    for (int w = 0; w < 8; ++w) v += sums[w][threadIdx.x];
    v = total == 0.0f ? 0.0f : v / total;
    const int64_t at = t * a.o_st + hq * a.o_sh + threadIdx.x;
    if (a.dtype == QG_F16) static_cast<__half*>(a.out)[at] = __float2half_rn(v);
    else static_cast<__nv_bfloat16*>(a.out)[at] = __float2bfloat16_rn(v);
  }
  if (a.lse && threadIdx.x == 0)
    a.lse[(int64_t)t * a.heads_q + hq] = total == 0.0f ? -INFINITY : (top + log2f(total)) * 0.69314718056f;
}

size_t prefix_bytes(int64_t B) { return (size_t)((B + 1) * 4 + 15) / 16 * 16; }

template <int G, int NT>
qg_status launch(const Attn4& a, void* workspace, cudaStream_t s) {
  constexpr int D = 64 * G;
  constexpr int kRing = kWarps * kStages * 2 * kChunk * (D / 2 + 4 * G);
  static PerDeviceOnce once;
  const qg_status st = once.run([](int) {
    return check_cuda(cudaFuncSetAttribute(attention_kv4_decode<G, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                           kRing + (4096 + 1) * 4),
                      "attention_kv4 shared memory");
  });
  if (st != QG_OK) return st;
  int32_t* prefix = static_cast<int32_t*>(workspace);
  float* parts = reinterpret_cast<float*>(static_cast<char*>(workspace) + prefix_bytes(a.B));
  const int grid = sm_count();
  LaunchCfg lc((unsigned)grid, 32 * kWarps, kRing + (a.B + 1) * 4, s);
  cudaError_t e = cudaLaunchKernelEx(&lc.cfg, attention_kv4_decode<G, NT>, a, prefix, parts);
  if (e != cudaSuccess) return check_cuda(e, "attention_kv4 decode launch");
  LaunchCfg lj(8 * NT, 256, 0, s);
  lj.cfg.gridDim.y = (unsigned)a.cache.heads;
  lj.cfg.gridDim.z = (unsigned)a.B;
  e = cudaLaunchKernelEx(&lj.cfg, attention_kv4_join<D>, a, (const int32_t*)prefix, (const float*)parts, grid * kWarps, NT);
  return check_cuda(e, "attention_kv4 join launch");
}

}  // namespace

size_t attention_kv4_decode_workspace(int64_t B, int64_t dim, int nt) {
  return prefix_bytes(B) + (size_t)2 * sm_count() * kWarps * part_floats(nt, (int)dim) * sizeof(float);
}

qg_status launch_attention_kv4_decode(const Attn4& a, int nt, void* workspace, cudaStream_t s) {
  if (a.cache.dim == 64) return nt == 1 ? launch<1, 1>(a, workspace, s) : launch<1, 2>(a, workspace, s);
  return nt == 1 ? launch<2, 1>(a, workspace, s) : launch<2, 2>(a, workspace, s);
}

}  // namespace qg
