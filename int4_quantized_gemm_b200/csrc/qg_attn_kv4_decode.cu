// qg_attn_kv4_decode.cu -- attention of few query rows over the paged 4-bit
// cache: every (sequence, KV head) whose query tokens times head group make at
// most 16 rows (single-token decode, draft tokens).
//
// Memory-bound in principle: a key and value of 128 channels are 144 bytes, so
// at HBM rate an SM has about 6 cycles for the 256 codes of a token.  What
// decides the time is therefore the instructions per code, and the codes are
// never dequantized one by one:
//   score_j = sum_g [ s_jg (q_g . c_jg) + o_jg sum(q_g) ]
//   out     = sum_j (p_j s_jg) (c_j - 8) + sum_j p_j (o_jg + 8 s_jg)
// (g: group of 64 channels; s, o: its scale and offset; c: codes).  The products
// run on the codes themselves.  A nibble masked into the low bits of a half is
// the fp16 subnormal c 2^-24 (or, four bits up, 16 c 2^-24), exact on the tensor
// cores: two codes cost one mask, with one shift per four.  Queries are scaled
// by a power of two to fp16 (1/16 of it where they meet a nibble four bits up),
// scale and offset enter per token and group in binary32.  p s is rounded to
// fp16 under a power of two kappa (a shift of the running maximum) that keeps
// s kappa near 2^4 at p = 1, 2^18 above the first fp16 subnormal, for the largest
// finite s that the row has seen: a later token's large or NaN scale costs no
// row digits that does not see it (one kappa for all rows was 1.5 % faster with
// one row tile, the same with two).  Codes are
// taken from their middle because values have either sign: without it the sum
// over n keys is large against the result and its truncation shows (0.0013
// relative error at 131071 keys): an exact fp16 addition of -8 2^-24 to each
// pair.
//
// mma.m16n8k16 with keys (16 tokens) or channels (16 of V^T) as its rows and up
// to 8 query rows as its columns: the accumulators of q.c and of the output
// have the same columns in the same lanes, and movmatrix turns the
// probabilities into the second product's operand.  (tcgen05 would take the
// codes through shared or tensor memory: more bytes moved per code than this
// has instructions.)  The maximum that scores are taken against moves only when
// 32 keys pass it by 8 binary digits: a vote instead of a reduction, and 32 keys
// at a time keep a warp's state small.
//
// Measured, 64 sequences of 4096..8192 tokens, 64/8 heads of 128: 122 us, HBM's
// rate is 70.  A product takes the sub-core's issue for 8 cycles, in which no
// other instruction goes out (probe: 8 products and 32 logic operations take 99
// cycles, 64 and 64 alone), so 16 keys of 128 channels cost 16 products x 8 and
// about 380 others (counted), 87 us of issue.  That is why the middle is an
// addition and not the other half of the products' depth (24 products: 7 us
// more).  About 12 us of a call are its beginning and end (lengths, first loads,
// joins).  The rest, about 20, is latency: three warps a scheduler are ready to
// issue 0.83 at a time, each a chain of load, product, vote, exponential, product.
//
// Every warp is a worker of its own: the chunks of tokens of all sequences
// and heads form one list, split evenly over the warps of one CTA per SM, so
// ragged lengths balance.  A warp streams its share through a ring of
// bulk copies (one per page piece and array) without any block barrier.  A
// (sequence, head) that one warp covers is written at once; parts are joined
// in list order, first those of one CTA by the CTA, then those that cross CTAs
// by a second kernel (no atomics: the same call gives the same bits).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "qg_device.cuh"
#include "qg_internal.h"
#include "qg_kv4_join.cuh"

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

// The ring: 64 tokens a stage and 2 stages for each of 12 warps (221 KB at 128 channels, the registers' 168 a thread).
// 64 sequences of 4096..8192 tokens, 64/8 heads of 128: 122 us (3.8 TB/s); 8 or 10 warps were 13 and 22 longer, stages
// of 32 tokens 16.  Heads of 64 take 128 registers: 16 warps 71 us, 12 warps 6 more.  Two row tiles take 208 and more: 2 x
// 131071 tokens, 4 new ones, 32/8 heads of 64: 76 us with 8 warps, not less with 12.
constexpr int kChunk = 64;   // tokens per ring stage
template <int G, int NT>
constexpr int kWarpsOf = NT == 2 ? 8 : G == 1 ? 16 : 12;  // workers per CTA (registers: 65536 / (32 workers))
constexpr int kStages = 2;
constexpr float kAhead = 8.0f;  // log2 of how far a score may pass the maximum it is taken against
constexpr uint32_t kMinus8 = 0x80088008u, kMinus128 = 0x80808080u;  // fp16x2: -8 2^-24, -128 2^-24 (16 codes' middle)

// log2 kappa before any scale is known: that of the subnormal ones.  The largest scale (fp16 bits) that a kappa holds.
constexpr float kLeastLift = 17.0f;
__device__ __forceinline__ uint32_t scale_limit(float lift) { return min((uint32_t)(21.0f - lift) << 10, 0x7BFFu); }

// device status sites
enum : uint32_t { kSiteSequence = 1, kSitePage = 2, kSiteWait = 3, kSiteCopy = 4 };

__device__ __forceinline__ void report(uint32_t code, uint32_t site) {
  atomicCAS(&g_status_attn, 0ull,
            (unsigned long long)code | ((unsigned long long)site << 8) | ((unsigned long long)blockIdx.x << 24));
}

__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The same with a zero accumulator.
__device__ __forceinline__ void mma16816_zero(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                              uint32_t b0, uint32_t b1) {
  asm(
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

__device__ __forceinline__ uint32_t add_halves(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("add.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t a) {
  uint32_t d;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
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
__device__ __forceinline__ void lds(uint32_t (&r)[N], const uint8_t* p) {
  static_assert(N == 1 || N == 2 || N == 4, "");
  if constexpr (N == 1) {
    r[0] = *reinterpret_cast<const uint32_t*>(p);
  } else if constexpr (N == 2) {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    r[0] = v.x, r[1] = v.y;
  } else {
    const uint4 v = *reinterpret_cast<const uint4*>(p);
    r[0] = v.x, r[1] = v.y, r[2] = v.z, r[3] = v.w;
  }
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
  s.lo = attn4_oldest(a, s.len - s.n);
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

// n units over `over` takers, the first n % over of them one more.
struct Share {
  uint32_t q, r;
  __device__ __forceinline__ Share(uint32_t n, uint32_t over) : q(n / over), r(n - n / over * over) {}
  __device__ __forceinline__ uint32_t first(uint32_t i) const { return q * i + min(i, r); }
  __device__ __forceinline__ uint32_t taker(uint32_t unit) const {
    return unit < (q + 1) * r ? unit / (q + 1) : r + (unit - (q + 1) * r) / q;
  }
};

// A part of a (sequence, head): rows of dim sums, then (log2 of the maximum, l) of each row.
__host__ __device__ constexpr int part_floats(int nt, int dim) { return 8 * nt * (dim + 2); }

// What crosses from a CTA into the next ones: the join kernel's work.
struct Crossing {
  int first, n, h, ctas;  // the sequence's first query and their number; ctas: how many the item spans from this one, 0: none
};

// Parts of the two levels and the crossings, in the workspace.
struct Scratch {
  Crossing* crossing;  // [grid]
  float* warp_parts;   // [grid * kWarps][2]: a continued item, an unfinished one
  float* cta_parts;    // [grid][2]
};

template <int D, int NT>
__device__ __forceinline__ const float2* part_head(const float* p, int row) {
  return reinterpret_cast<const float2*>(p + 8 * NT * D + 2 * row);
}

template <int D, int NT>
__device__ __forceinline__ void write_part(float* p, int row, int lane, float top, float l, const float (&v)[D / 32]) {
  if constexpr (D == 128) *reinterpret_cast<float4*>(p + row * D + 4 * lane) = make_float4(v[0], v[1], v[2], v[3]);
  else *reinterpret_cast<float2*>(p + row * D + 2 * lane) = make_float2(v[0], v[1]);
  if (lane == 0) *reinterpret_cast<float2*>(p + 8 * NT * D + 2 * row) = make_float2(top, l);
}

template <int G, int NT>
__global__ void __launch_bounds__(32 * kWarpsOf<G, NT>, 1)
    attention_kv4_decode(const __grid_constant__ Attn4 a, const __grid_constant__ Scratch scratch) {
  constexpr int kWarps = kWarpsOf<G, NT>;
  constexpr int D = 64 * G;
  constexpr uint32_t kCodes = kChunk * D / 2, kParams = kChunk * G * 4;
  constexpr uint32_t kStage = 2 * (kCodes + kParams);
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ __align__(8) uint64_t bars[kWarps][kStages];
  __shared__ int warp_sums[kWarps];
  // a warp's parts: of an item that another worker started (1: goes on behind this worker, 2: ends here), and of
  // one that starts here and goes on
  struct Left {
    int head, head_first, head_n, head_h, tail, tail_first, tail_n, tail_h, tail_last;
  };
  __shared__ Left left[kWarps];
  int* prefix = reinterpret_cast<int*>(smem);  // before the ring is used

  const int tid = threadIdx.x, lane = tid & 31, warp = tid / 32;
  const int q4 = lane & 3, r8 = lane >> 2;
  if (lane == 0) {
#pragma unroll
    for (int i = 0; i < kStages; ++i) mbar_init(smem_u32(&bars[warp][i]), 1);
    fence_mbar_init();
  }
  pdl_trigger();
  // (Also behind the prompt kernel of the same call, with which it shares nothing but its inputs: only this wait makes
  // what earlier grids wrote visible.  Overlapped without it, 16 sequences of 4096 tokens, two with 512 new ones, took
  // 112 instead of 122 us.)
  pdl_wait();

  // prefix[b]: chunks (times heads) of the sequences before b
  const int per = (a.B + 32 * kWarps - 1) / (32 * kWarps);
  {
    int sum = 0;
#pragma unroll 1
    for (int b = tid * per; b < min(a.B, (tid + 1) * per); ++b) {
      bool ok;
      const int units = sequence<NT>(a, b, ok).chunks * a.cache.heads;
      if (!ok && blockIdx.x == 0) report(kDevBadArg, kSiteSequence);
      prefix[b] = units;
      sum += units;
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
#pragma unroll 1
    for (int b = tid * per; b < min(a.B, (tid + 1) * per); ++b) {
      const int units = prefix[b];
      prefix[b] = at;
      at += units;
      if (b == a.B - 1) prefix[a.B] = at;
    }
    __syncthreads();
  }
  // the list's units over the CTAs, a CTA's over its warps
  const Share ctas((uint32_t)prefix[a.B], gridDim.x);
  const uint32_t cta0 = ctas.first(blockIdx.x);
  const Share warps(ctas.first(blockIdx.x + 1) - cta0, kWarps);
  const int u0 = (int)(cta0 + warps.first(warp)), units = (int)(warps.first(warp + 1) - warps.first(warp));
  const bool alone = warps.q == 0 && warps.r == 1;  // the CTA's one worker: its parts are the CTA's
  if (lane == 0) left[warp].head = left[warp].tail = 0;

  Cursor<NT> fill = {};
  if (units > 0) {
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
  __syncthreads();  // the prefix has been read: its place is the ring's
  fence_proxy_async_smem();

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
      const int i = (int)kv4_page(a.cache, (uint32_t)t >> 4);  // t / P
      in_page = t - i * P;
      page = a.table[(int64_t)fill.b * a.table_ld + i];
      if (page < 0 || page >= a.cache.pages) {
        report(kDevBadArg, kSitePage);
        page = -1;
      } else if (!dcheck(in_area(in_page, piece, P) && in_area(dst_off, bytes, kStage) && (dst_off | bytes) % 16 == 0,
                         &g_status_attn, kSiteCopy)) {
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

  // --- the item in hand -------------------------------------------------------
  uint32_t qf[NT][G][2][4];        // queries, the second operand of q . c
  float qs[NT][2][G];              // sums of the group's queries, times 2^-24: columns 2 q4, 2 q4 + 1
  float sigma[NT][2];              // scale log2(e) 2^24 over the queries' power of two
  float m[NT][2], l[NT][2];        // the maximum that scores are taken against (before sigma), and the sum
  uint32_t unseen = 0;             // bit 2 nt + c: no key seen yet, m is 0
  bool fresh = false;              // any column of the warp is such
  float ob[NT][2][G];              // sum p o
  float o[NT][G][4][4];            // sum p s (c - 8) 2^-24
  int end[NT][2], beg[NT][2];      // visible keys of the columns
  float lift[NT][2];               // log2 kappa: l, ob and o hold p kappa
  uint32_t limit = 0;              // largest scale (fp16 bits) that every column's kappa holds
  bool starts_item = false;
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
      e = max(-120, min(100, e));
      const float up = __uint_as_float((uint32_t)(127 + e) << 23);
      // (not zero, which would make a NaN of a hidden score, and not so large that a score, 2^8 at most, leaves binary32:
      // from here on all of the weight is on the best key anyway)
      const float sg = fminf(
          fmaxf(a.scale * 1.44269504088896f * 16777216.0f * __uint_as_float((uint32_t)(127 - e) << 23), 0x1p-126f), 0x1p118f);
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
        m[nt][c] = 0.0f;
        lift[nt][c] = kLeastLift;
        l[nt][c] = 0.0f;
        const int col = nt * 8 + 2 * q4 + c;
        const int pos = s.len - s.n + min(col, rows - 1) / a.group;
        end[nt][c] = a.causal ? min(s.len, pos + 1) : s.len;
        beg[nt][c] = attn4_oldest(a, pos);
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
    limit = scale_limit(kLeastLift);
    unseen = (1u << (2 * NT)) - 1;
    fresh = true;
    starts_item = use.c == 0;
  };

  auto end_item = [&](bool whole) {
    const Seq& s = use.s;
    const int rows = s.n * a.group;
    float* part = alone ? scratch.cta_parts + (int64_t)(blockIdx.x * 2 + starts_item) * part_floats(NT, D)
                        : scratch.warp_parts + ((int64_t)(blockIdx.x * kWarps + warp) * 2 + starts_item) * part_floats(NT, D);
    if (!whole && lane == 0) {
      if (starts_item)
        left[warp].tail = 1, left[warp].tail_first = s.first, left[warp].tail_n = s.n, left[warp].tail_h = use.h,
        left[warp].tail_last = u0 + units - 1 + s.chunks - 1 - use.c;
      else
        left[warp].head = use.c + 1 == s.chunks ? 2 : 1, left[warp].head_first = s.first, left[warp].head_n = s.n,
        left[warp].head_h = use.h;
    }
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
        const float top = unseen >> (2 * nt + c) & 1 ? -INFINITY : m[nt][c] * sigma[nt][c] - lift[nt][c];  // log2 units
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

  // the token of fragment row r (0..7): pairs (0,1), (3,2), (4,5), (7,6), which spreads the value loads over the banks
  const int kt = r8 ^ ((r8 >> 1) & 1);
  const int vt0 = 2 * q4 + (q4 & 1), vt1 = vt0 ^ 1;  // rows 2 q4 and 2 q4 + 1
  uint32_t phases = 0;

  int filled = 0;          // chunks whose copies were issued
  bool new_item = true;
  if (units > 0) look_up();
#pragma unroll 1
  for (int i = 0; i < units; ++i) {
    const int stage = i % kStages;
#pragma unroll 1
    while (filled < units && filled < i + kStages) {  // stage (i - 1) % kStages has been read by the whole warp
      issue(filled % kStages);
      if (++filled < units) {
        fill.next(a);
        look_up();
      }
    }
    if (new_item) begin_item();
    if (!__all_sync(0xffffffffu, mbar_wait(smem_u32(&bars[warp][stage]), (phases >> stage) & 1, &g_status_attn, kSiteWait))) {
      // give up, all lanes together: let the other copies in flight land (bounded), then leave
      for (int k = 1; k < kStages && i + k < filled; ++k)
        mbar_wait(smem_u32(&bars[warp][(i + k) % kStages]), (phases >> ((i + k) % kStages)) & 1, &g_status_attn, kSiteWait);
      break;
    }
    phases ^= 1u << stage;
    const uint8_t* base = smem + (warp * kStages + stage) * kStage;
    const uint8_t *kc = base, *vc = base + kCodes, *kp = base + 2 * kCodes, *vp = kp + kParams;
    const int t0 = (use.s.c0 + use.c) * kChunk;
    auto tiles = [&](auto all) {  // all: every row sees every key
      constexpr bool kAll = decltype(all)::value;
#pragma unroll 1
      for (int step = 0; step < kChunk / 32; ++step) {  // two tiles of 16 keys
        float x[2][NT][4];
        uint32_t vw[2][2][G];
#pragma unroll
        for (int i2 = 0; i2 < 2; ++i2) {
          const int tile = 2 * step + i2;
          // scores, less the maximum (m sigma alone may be so large that its rounding passes the exponential's range)
          uint32_t kw[2][2 * G], pw[2][G];
#pragma unroll
          for (int hh = 0; hh < 2; ++hh) {
            const int tok = tile * 16 + hh * 8 + kt;
            lds(kw[hh], kc + tok * (D / 2) + q4 * (8 * G));
            lds(pw[hh], kp + tok * (G * 4));
            lds(vw[i2][hh], vp + tok * (G * 4));
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
          for (int k = 0; k < 4; ++k) {
            float2 so[G];
#pragma unroll
            for (int g = 0; g < G; ++g) so[g] = half2_f32(pw[k >> 1][g]);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              float v = fmaf(so[0].y, qs[nt][k & 1][0], -m[nt][k & 1]);
#pragma unroll
              for (int g = 0; g < G; ++g) {
                if (g > 0) v = fmaf(so[g].y, qs[nt][k & 1][g], v);
                v = fmaf(acc[nt][g][k], so[g].x, v);
              }
              if constexpr (!kAll) {
                const int t = t0 + tile * 16 + (k >> 1) * 8 + kt;
                if (t < beg[nt][k & 1] || t >= end[nt][k & 1]) v = -INFINITY;
              }
              x[i2][nt][k] = v;
            }
          }
        }

        // does a score pass the maximum too far, or a scale (of a key that any row sees) what a kappa holds?
        uint32_t smax = 0;
        float far[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) far[nt][0] = far[nt][1] = -INFINITY;
#pragma unroll
        for (int i2 = 0; i2 < 2; ++i2) {
#pragma unroll
          for (int hh = 0; hh < 2; ++hh) {
            const int t = t0 + (2 * step + i2) * 16 + hh * 8 + kt;
            if (kAll || (t >= use.s.lo && t < use.s.len)) {
#pragma unroll
              for (int g = 0; g < G; ++g) smax = max_halves(smax, vw[i2][hh][g]);
            }
          }
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int k = 0; k < 4; ++k) far[nt][k & 1] = fmaxf(far[nt][k & 1], x[i2][nt][k]);
        }
        smax &= 0x7FFFu;  // fp16 bits order like the values (a scale is not negative)
        bool move = fresh || smax > limit;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) move |= far[nt][0] * sigma[nt][0] > kAhead || far[nt][1] * sigma[nt][1] > kAhead;
        if (__any_sync(0xffffffffu, move)) {
          // the tokens' largest scales; one that is not finite makes a NaN under any kappa
          uint32_t scale[2][2], least = 0xFFFFFFFFu;
#pragma unroll
          for (int i2 = 0; i2 < 2; ++i2)
#pragma unroll
            for (int hh = 0; hh < 2; ++hh) {
              scale[i2][hh] = 0;
#pragma unroll
              for (int g = 0; g < G; ++g) {
                const uint32_t b = vw[i2][hh][g] & 0x7FFFu;
                if (b < 0x7C00u) scale[i2][hh] = max(scale[i2][hh], b);
              }
            }
          // the largest score and scale of the keys that each column's row sees (what others hold is nothing to it)
          float best[NT][2];
          uint32_t top[NT][2];
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              best[nt][c] = fmaxf(fmaxf(x[0][nt][c], x[0][nt][2 + c]), fmaxf(x[1][nt][c], x[1][nt][2 + c]));
              top[nt][c] = 0;
#pragma unroll
              for (int i2 = 0; i2 < 2; ++i2)
#pragma unroll
                for (int hh = 0; hh < 2; ++hh)
                  if (kAll || x[i2][nt][2 * hh + c] != -INFINITY) top[nt][c] = max(top[nt][c], scale[i2][hh]);
            }
#pragma unroll
          for (int d = 4; d < 32; d <<= 1)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int c = 0; c < 2; ++c) {
                best[nt][c] = fmaxf(best[nt][c], __shfl_xor_sync(0xffffffffu, best[nt][c], d));
                top[nt][c] = max(top[nt][c], __shfl_xor_sync(0xffffffffu, top[nt][c], d));
              }
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              const uint32_t bit = 1u << (2 * nt + c);
              const bool first = unseen & bit;
              float t = fmaxf(best[nt][c], first ? -INFINITY : 0.0f);  // how far the maximum moves
              if (t > -INFINITY) unseen &= ~bit;
              else t = 0.0f;
              m[nt][c] += t;
              // scale times kappa in [2^3, 2^4), up to 2^6 before this is done again; p up to 2^8
              const float old = lift[nt][c];
              if (top[nt][c] > scale_limit(old)) lift[nt][c] = 18.0f - (float)(top[nt][c] >> 10);  // the scale's exponent, 15 for 1
              least = min(least, scale_limit(lift[nt][c]));
              const float corr = first ? 0.0f : ex2(fmaf(-t, sigma[nt][c], lift[nt][c] - old));
#pragma unroll
              for (int i2 = 0; i2 < 2; ++i2)
#pragma unroll
                for (int k = c; k < 4; k += 2) x[i2][nt][k] -= t;
              l[nt][c] *= corr;
#pragma unroll
              for (int g = 0; g < G; ++g) {
                ob[nt][c][g] *= corr;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                  o[nt][g][k][c] *= corr;
                  o[nt][g][k][2 + c] *= corr;
                }
              }
            }
          fresh = __any_sync(0xffffffffu, unseen != 0);
          limit = __reduce_min_sync(0xffffffffu, least);
        }

        // probabilities (times kappa) and the second product
#pragma unroll
        for (int i2 = 0; i2 < 2; ++i2) {
          const int tile = 2 * step + i2;
          uint32_t pf[NT][G][2];
#pragma unroll
          for (int hh = 0; hh < 2; ++hh) {
            float2 so[G];
#pragma unroll
            for (int g = 0; g < G; ++g) {
              so[g] = half2_f32(vw[i2][hh][g]);
              so[g].y = fmaf(8.0f, so[g].x, so[g].y);
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              float p[2];
#pragma unroll
              for (int c = 0; c < 2; ++c) {
                p[c] = ex2(fmaf(x[i2][nt][2 * hh + c], sigma[nt][c], lift[nt][c]));
                l[nt][c] += p[c];
              }
#pragma unroll
              for (int g = 0; g < G; ++g) {
                float ps[2];
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                  if (kAll || x[i2][nt][2 * hh + c] != -INFINITY) {  // a hidden key's params may be anything
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
              const uint32_t e0 = __byte_perm(v0[0][g], v1[0][g], sel), e1 = __byte_perm(v0[1][g], v1[1][g], sel);
              const uint32_t f0 = e0 >> 8, f1 = e1 >> 8;
              // codes from their middle, exact
              const uint32_t a0 = add_halves(e0 & 0x000F000Fu, kMinus8), a1 = add_halves(f0 & 0x000F000Fu, kMinus8);
              const uint32_t a2 = add_halves(e1 & 0x000F000Fu, kMinus8), a3 = add_halves(f1 & 0x000F000Fu, kMinus8);
              const uint32_t b0 = add_halves(e0 & 0x00F000F0u, kMinus128), b1 = add_halves(f0 & 0x00F000F0u, kMinus128);
              const uint32_t b2 = add_halves(e1 & 0x00F000F0u, kMinus128), b3 = add_halves(f1 & 0x00F000F0u, kMinus128);
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) {
                mma16816(o[nt][g][2 * half], a0, a1, a2, a3, pf[nt][g][0], pf[nt][g][1]);
                mma16816(o[nt][g][2 * half + 1], b0, b1, b2, b3, pf[nt][g][0], pf[nt][g][1]);
              }
            }
          }
        }
      }
    };
    if (t0 >= max_beg && t0 + kChunk <= min_end) tiles(std::true_type{});
    else tiles(std::false_type{});

    __syncwarp();
    // the item's end, or the worker's
    new_item = use.c + 1 == use.s.chunks;
    if (new_item || i + 1 == units) end_item(new_item && starts_item);
    if (i + 1 < units) use.next(a);
  }

  // --- what the warps left unfinished -----------------------------------------
  // In list order: each warp's continued item, then the one it started.  A group of parts that belong together
  // begins with a started item (or the CTA's first part) and takes every continued one up to the item's end.
  __syncthreads();
  const float* base = scratch.warp_parts + (int64_t)blockIdx.x * kWarps * 2 * part_floats(NT, D);
  // bit w: warp w's head, a head that ends its item, a tail
  const int kind = lane < kWarps ? left[lane].head : 0;
  const uint32_t heads = __ballot_sync(0xffffffffu, kind != 0), done = __ballot_sync(0xffffffffu, kind == 2);
  const uint32_t tails = __ballot_sync(0xffffffffu, lane < kWarps && left[lane].tail != 0);
  // groups: the first warp's head (if it goes on from another CTA), and every tail; their rows go round the warps
  const uint32_t starts_at = tails << 1 | (heads & 1);  // bit 0: that head, bit w + 1: warp w's tail
  const int last = 31 - __clz(tails);                   // the only item that can leave the CTA starts here
  const bool crosses = tails != 0 && (done >> (last + 1)) == 0;
  if (tid == 0) {
    Crossing cross = {0, 0, 0, 0};
    if (crosses)
      cross = {left[last].tail_first, left[last].tail_n, left[last].tail_h,
               (int)(ctas.taker(left[last].tail_last) - blockIdx.x) + 1};
    scratch.crossing[blockIdx.x] = cross;
  }
  if (alone) return;
  int unit = 0;
#pragma unroll 1
  for (uint32_t todo = starts_at; todo; todo &= todo - 1) {
    const int k = __ffs(todo) - 1;
    const bool starts = k > 0;
    const int w0 = starts ? k - 1 : 0;  // the group's first part is this warp's
    // the heads that follow: up to the first that ends the item, all of them without a gap
    const uint32_t after = heads >> (w0 + 1), stop = done >> (w0 + 1);
    bool ends = !starts && (done & 1);
    int count = 1;
    if (!ends) {
      const int run = __ffs(~after) - 1, until = stop ? __ffs(stop) : 33;
      ends = until <= run;
      count += min(run, until);
    }
    const int first = starts ? left[w0].tail_first : left[w0].head_first, h = starts ? left[w0].tail_h : left[w0].head_h;
    const int rows = (starts ? left[w0].tail_n : left[w0].head_n) * a.group;
#pragma unroll 1
    for (int row = (warp + kWarps - unit % kWarps) % kWarps; row < rows; row += kWarps) {
      float v[D / 32], top, l;
      const auto part = [&](int i) { return base + (int64_t)(i == 0 ? 2 * w0 + starts : 2 * (w0 + i)) * part_floats(NT, D); };
      add_parts<D>([&](int i) { return part(i) + row * D; }, [&](int i) { return part_head<D, NT>(part(i), row); }, count,
                   lane, top, l, v);
      if (starts && ends) write_row<D>(a, first, h, row, lane, top, l, v);
      else
        write_part<D, NT>(scratch.cta_parts + (int64_t)(blockIdx.x * 2 + starts) * part_floats(NT, D), row, lane, top, l, v);
    }
    unit += rows;
  }
}

// Joins the parts of the (sequence, head)s that cross CTAs: block (8 rows, CTA in which it starts), a warp per row.
template <int D, int NT>
__global__ void __launch_bounds__(256)
    attention_kv4_join(const __grid_constant__ Attn4 a, const __grid_constant__ Scratch scratch) {
  pdl_trigger();
  pdl_wait();
  const int cta = blockIdx.y, lane = threadIdx.x & 31, row = blockIdx.x * 8 + threadIdx.x / 32;
  const Crossing c = scratch.crossing[cta];
  if (c.ctas == 0 || row >= c.n * a.group) return;
  float v[D / 32], top, l;
  const auto part = [&](int k) { return scratch.cta_parts + (int64_t)((cta + k) * 2 + (k == 0)) * part_floats(NT, D); };
  add_parts<D>([&](int k) { return part(k) + row * D; }, [&](int k) { return part_head<D, NT>(part(k), row); }, c.ctas, lane,
               top, l, v);
  write_row<D>(a, c.first, c.h, row, lane, top, l, v);
}

size_t crossing_bytes() { return (size_t)sm_count() * sizeof(Crossing); }

template <int G, int NT>
Scratch scratch_of(void* workspace) {
  Scratch s;
  s.crossing = static_cast<Crossing*>(workspace);
  s.warp_parts = reinterpret_cast<float*>(static_cast<char*>(workspace) + crossing_bytes());
  s.cta_parts = s.warp_parts + (int64_t)sm_count() * kWarpsOf<G, NT> * 2 * part_floats(NT, 64 * G);
  return s;
}

template <int G, int NT>
qg_status launch(const Attn4& a, void* workspace, cudaStream_t s) {
  constexpr int D = 64 * G, kWarps = kWarpsOf<G, NT>;
  constexpr int kRing = kWarps * kStages * 2 * kChunk * (D / 2 + 4 * G);
  constexpr int kMost = kRing > 4097 * 4 ? kRing : 4097 * 4;  // the prefix of 4096 sequences shares the ring's place
  static PerDeviceOnce once;
  const qg_status st = once.run([](int) {
    return check_cuda(cudaFuncSetAttribute(attention_kv4_decode<G, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, kMost),
                      "attention_kv4 shared memory");
  });
  if (st != QG_OK) return st;
  const int grid = sm_count();
  const Scratch scratch = scratch_of<G, NT>(workspace);
  LaunchCfg lc((unsigned)grid, 32 * kWarps, kMost, s);
  cudaError_t e = cudaLaunchKernelEx(&lc.cfg, attention_kv4_decode<G, NT>, a, scratch);
  return check_cuda(e, "attention_kv4 decode launch");
}

template <int G, int NT>
qg_status launch_join(const Attn4& a, void* workspace, cudaStream_t s) {
  const Scratch scratch = scratch_of<G, NT>(workspace);
  LaunchCfg lc(NT, 256, 0, s);
  lc.cfg.gridDim.y = (unsigned)sm_count();
  return check_cuda(cudaLaunchKernelEx(&lc.cfg, attention_kv4_join<64 * G, NT>, a, scratch), "attention_kv4 join launch");
}

}  // namespace

size_t attention_kv4_decode_workspace(int64_t dim, int nt) {
  return crossing_bytes() + (size_t)sm_count() * ((nt == 2 ? kWarpsOf<2, 2> : dim == 64 ? kWarpsOf<1, 1> : kWarpsOf<2, 1>) + 1) * 2 * part_floats(nt, (int)dim) * sizeof(float);
}

qg_status launch_attention_kv4_decode(const Attn4& a, int nt, void* workspace, cudaStream_t s) {
  if (a.cache.dim == 64)
    return nt == 1 ? launch<1, 1>(a, workspace, s) : launch<1, 2>(a, workspace, s);
  return nt == 1 ? launch<2, 1>(a, workspace, s) : launch<2, 2>(a, workspace, s);
}

qg_status launch_attention_kv4_decode_join(const Attn4& a, int nt, void* workspace, cudaStream_t s) {
  if (a.cache.dim == 64) return nt == 1 ? launch_join<1, 1>(a, workspace, s) : launch_join<1, 2>(a, workspace, s);
  return nt == 1 ? launch_join<2, 1>(a, workspace, s) : launch_join<2, 2>(a, workspace, s);
}

}  // namespace qg
