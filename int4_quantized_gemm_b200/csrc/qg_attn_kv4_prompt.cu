// qg_attn_kv4_prompt.cu -- attention of many query rows over the paged 4-bit
// cache: (sequence, KV head)s with more query tokens times head group than the
// decode kernel takes (prompts, chunks of prompts, long drafts).
//
// Compute-bound: 4 dim operations and one exponential per (row, key).  One CTA
// takes 256 rows (two tiles of 128, so that both share a step's dequantized keys
// and values) of a (sequence, KV head) and walks over the keys 64 at a time:
//   2 MMA warps      one per row tile; tcgen05: S = Q K^T (M 128, N 64, K dim)
//                    and O += P V (P from tensor memory, N dim), accumulators in
//                    tensor memory: 2 x 2 x 64 columns S, 2 x dim columns O
//   2 loader warps   packed codes and params of 64 tokens a stage, bulk copies,
//                    keys and values in rings of their own
//   2 x 4 warps      softmax of a row tile, a thread per row: maximum, p =
//                    2^(x - m), P in fp16 over S's columns
//   2 x 4 warps      codes -> fp16 (c s + o, one rounding) into the swizzled
//                    K-major operands K [key][channel] and V^T [channel][key]
// Scores of a row tile alternate between two places in tensor memory and run
// two steps ahead, so its softmax does not wait for the products of its own
// probabilities.  The maximum that scores are taken against moves only when a
// row passes it by 8 binary digits, so the accumulator is rarely rescaled; p
// carries a factor 2^7 that keeps small ones out of fp16's subnormals (p 2^7 <
// 2^15).
//
// Roundings to fewer than 32 bits, all to fp16 because the tensor cores take two
// 16-bit operands: queries (exact for fp16; bf16 has fewer digits and is scaled
// into fp16's range, each row by its own power of two), a key's and a value's c s + o, and p.  Each is half a step
// of 2^-11; scores, maxima, sums and outputs are binary32.  (At 2 x 4096 tokens
// of fp16 they make 0.00037 of relative error beside the output's own rounding
// of 0.00021: keys 0.00027, values 0.00020, p 0.00015.  Splitting keys into two
// operands would take the first away for 1.4 times the tensor cores' time.)
//
// 2 x 4096 tokens, 32 heads of 128, causal: 345 us in a row of 30 calls, 368 in
// seconds of them, when the power limit lowers the clock (0.80 and 0.75 PFLOP/s).
// A step of 64 keys by 256 rows takes about 2250 cycles.  The tensor cores hold
// products for 1590 of them, of which 1020 are arithmetic (a product of N 64 reads
// both operands from shared memory and takes 65 cycles instead of 32);
// exponentials need 1024 of the MUFU.  The two tiles share both units in phase,
// which leaves the rest.  Tried and slower: scores of 128 keys
// at once (one place for S, 419 us), tiles taking turns at the tensor cores
// (390), two threads a row, 16 warps of softmax (396), the maximum beside the
// exponentials of a stale one (361), a part of the exponentials as polynomials.
//
// Channels of K and Q lie in the order 0 4 1 5 2 6 3 7 of each 8 (the order in
// which masks take nibbles from a word); row 8 i + j of a V^T group is channel
// 8 j + i, which spreads the stores over the banks; the epilogue puts the
// output's columns back.
//
// With few (rows, head)s the keys are split over CTAs whose parts a second
// kernel joins in order (16 sequences of 4096 tokens, two with 64 new tokens: 75
// us, 33 more without).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "qg_device.cuh"
#include "qg_internal.h"
#include "qg_kv4_join.cuh"

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

constexpr int kRows = 256;      // query rows per CTA, two tiles of 128
constexpr int kKeys = 64;       // keys per step
constexpr int kBuf = 4;         // buffers of dequantized keys and values
constexpr int kRaw = 3;         // raw stages
constexpr int kThreads = 640;
// Registers a thread: 96 at launch (65536 / 640); then 144 for the softmax warps, 72 for the warps that dequantize and
// 48 for the others: 256 * 144 + 256 * 72 + 128 * 48 = 640 * 96.
constexpr int kLaunchRegs = 96, kSoftmaxRegs = 144, kDequantRegs = 72, kOtherRegs = 48;
static_assert(256 * kSoftmaxRegs + 256 * kDequantRegs + 128 * kOtherRegs <= kThreads * kLaunchRegs, "");
// Warps 0 and 1 issue the products of a row tile each, 2 and 3 load keys and values.  (One warp for both tiles spent
// half of its time between the products, in waits whose barriers had long completed.)
constexpr int kMmaWarp = 0, kLoadWarp = 2, kSoftmaxWarp = 4, kKeyWarp = 12, kValueWarp = 16;
constexpr float kLift = 7.0f, kAhead = 8.0f;
constexpr float kFarScore = 8192.0f;  // log2 units

enum : uint32_t {
  kSiteSequence = 1, kSitePage, kSiteRawFull, kSiteRawEmpty, kSiteKFull, kSiteKEmpty, kSiteVFull, kSiteVEmpty,
  kSiteS, kSiteP, kSiteO, kSiteQ, kSiteDrain, kSiteCopy
};

__device__ __forceinline__ void report(uint32_t code, uint32_t site) {
  atomicCAS(&g_status_prompt, 0ull,
            (unsigned long long)code | ((unsigned long long)site << 8) | ((unsigned long long)blockIdx.x << 24));
}

__device__ __forceinline__ uint32_t h2_fma(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t d;
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
  return d;
}
__device__ __forceinline__ uint32_t h2_add(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("add.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
// each half held to +-65504; a NaN becomes 65504
__device__ __forceinline__ uint32_t h2_finite(uint32_t a) {
  uint32_t d;
  asm("min.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(0x7BFF7BFFu));
  asm("max.f16x2 %0, %0, %1;" : "+r"(d) : "r"(0xFBFFFBFFu));
  return d;
}

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst), "l"(src),
      "r"(bytes), "r"(bar)
      : "memory");
}

// True on one lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.b32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
}

// D = A B and D += A B, one K step; the second with A in tensor memory too.
__device__ __forceinline__ void mma_first(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, 0, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d), "l"(a), "l"(b), "r"(idesc)
      : "memory");
}
__device__ __forceinline__ void mma_next(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, 1, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d), "l"(a), "l"(b), "r"(idesc)
      : "memory");
}
__device__ __forceinline__ void mma_next_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, 1, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d), "r"(a), "l"(b), "r"(idesc)
      : "memory");
}

__device__ __forceinline__ void sts128(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}

// Codes of nibbles 0..3 of each half of w as fp16 pairs 0 (nibble 0 of both halves) .. 3, exact
__device__ __forceinline__ void codes_f16(uint32_t w, uint32_t (&c)[4]) {
  const uint32_t w8 = w >> 8;
  c[0] = h2_add((w & 0x000F000Fu) | 0x64006400u, 0xE400E400u);                  // 1024 + c, less 1024
  c[1] = h2_fma((w & 0x00F000F0u) | 0x64006400u, 0x2C002C00u, 0xD400D400u);     // (1024 + 16 c) / 16 - 64
  c[2] = h2_add((w8 & 0x000F000Fu) | 0x64006400u, 0xE400E400u);
  c[3] = h2_fma((w8 & 0x00F000F0u) | 0x64006400u, 0x2C002C00u, 0xD400D400u);
}

// Does any of a stage's params (words of 4 bytes, for the whole warp to look at) give a value that is not a finite
// fp16: not finite itself, or its largest code's value beyond the type?
template <int WORDS>
__device__ __forceinline__ bool any_odd(const uint8_t* params, int lane) {
  static_assert(WORDS % 64 == 0, "");
  uint32_t most = 0;  // the largest magnitudes; NaN if one is
#pragma unroll
  for (int i = 0; i < WORDS / 64; ++i) {
    const uint2 w = *reinterpret_cast<const uint2*>(params + (i * 32 + lane) * 8);
    const uint32_t top = h2_fma(__byte_perm(w.x, w.y, 0x5410), 0x4B804B80u, __byte_perm(w.x, w.y, 0x7632)) & 0x7FFF7FFFu;
    asm("max.NaN.f16x2 %0, %0, %1;" : "+r"(most) : "r"(top));
  }
  return __any_sync(0xffffffffu, (most & 0x7C00u) == 0x7C00u || (most & 0x7C000000u) == 0x7C000000u);
}
__device__ __forceinline__ bool not_finite(uint32_t p) {
  return (p & 0x7C00u) == 0x7C00u || (p & 0x7C000000u) == 0x7C000000u;
}

struct Job {
  int b, h, tile;             // sequence, KV head, 256-row tile
  int split;                  // share of the keys
  int first, n, len, rows;    // the sequence
};

// Shares of the keys: as many as there are SMs for the (row tile, head)s, at most 32.
__host__ __device__ __forceinline__ int key_splits(int64_t tiles, int64_t heads, int sms) {
  const int64_t n = sms / (tiles * heads > 1 ? tiles * heads : 1);
  return n < 1 ? 1 : n > 32 ? 32 : (int)n;
}

__device__ __forceinline__ int tiles_of(const Attn4& a, int b, int min_rows) {
  int first, n, len;
  attn4_sequence(a, b, first, n, len);
  return n * a.group >= min_rows ? (n * a.group + kRows - 1) / kRows : 0;
}

// The shares of the keys of each of the call's tiles: the row counts of a ragged call are on the device.
__device__ __forceinline__ int splits_of(const Attn4& a, int min_rows, int sms, int lane) {
  if (!a.q_starts) return key_splits((int64_t)a.B * ((a.n_uniform * a.group + kRows - 1) / kRows), a.cache.heads, sms);
  int tiles = 0;
#pragma unroll 4
  for (int b = lane; b < a.B; b += 32) tiles += tiles_of(a, b, min_rows);
  return key_splits(__reduce_add_sync(0xffffffffu, tiles), a.cache.heads, sms);
}

// Which rows a block works on, in blocks of (tile, split, head); a sequence's tiles in descending order, so that a
// causal mask's longest start first.
__device__ __forceinline__ bool find_job(const Attn4& a, int min_rows, int splits, int block, int lane, Job& j) {
  j.h = block % a.cache.heads;
  block /= a.cache.heads;
  j.split = block % splits;
  block /= splits;
  if (!a.q_starts) {
    const int per = (a.n_uniform * a.group + kRows - 1) / kRows;
    j.b = block % a.B;
    j.tile = per - 1 - block / a.B;
    if (j.tile < 0) return false;
  } else {
    int base = 0, at = 0;
    j.b = -1;
    for (; base < a.B; base += 32) {  // the whole warp
      const int tiles = base + lane < a.B ? tiles_of(a, base + lane, min_rows) : 0;
      int scan = tiles;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, scan, d);
        if (lane >= d) scan += v;
      }
      const uint32_t found = __ballot_sync(0xffffffffu, block < at + scan);
      if (found) {
        const int src = __ffs(found) - 1;
        j.b = base + src;
        const int before = at + __shfl_sync(0xffffffffu, scan - tiles, src);
        j.tile = __shfl_sync(0xffffffffu, tiles, src) - 1 - (block - before);
        break;
      }
      at += __shfl_sync(0xffffffffu, scan, 31);
    }
    if (j.b < 0) return false;
  }
  attn4_sequence(a, j.b, j.first, j.n, j.len);
  j.rows = j.n * a.group;
  return true;
}

template <int G>
struct Layout {
  static constexpr int D = 64 * G;
  static constexpr uint32_t kBlock = 128 * 128;                 // 128 rows of 128 bytes
  static constexpr uint32_t kOperand = G * kBlock;              // 128 x D fp16
  static constexpr uint32_t kStep = kKeys * D * 2;              // a step's keys or values
  static constexpr uint32_t q = 0;                              // [2 tiles] [G][128 rows][64 channels]
  static constexpr uint32_t k = 2 * kOperand;                   // [kBuf] [G][64 keys][64 channels]
  static constexpr uint32_t v = k + kBuf * kStep;               // [kBuf] [D rows][64 keys]
  // stages of 64 tokens: keys' codes and params and the values' params; values' codes and params
  static constexpr uint32_t kCodes = kKeys * D / 2, kParams = kKeys * G * 4;
  static constexpr uint32_t kKeyStage = kCodes + 2 * kParams, kValueStage = kCodes + kParams;
  static constexpr uint32_t keys = v + kBuf * kStep, values = keys + kRaw * kKeyStage;
  static constexpr uint32_t bytes = values + kRaw * kValueStage;
};

// The softmax warps wait for the exponents that the warps of the values' dequantization take.
__device__ __forceinline__ void exponents_barrier() { named_barrier(1, 256 + 128); }

template <int N>
__device__ __forceinline__ void regs_up() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_down() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// The largest of a row's 64 scores (kAll: all of them, else columns [cb, ce)).
template <bool kAll>
__device__ __forceinline__ float row_max(const uint32_t (&v)[2][32], int cb, int ce) {
  float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
  for (int c = 0; c < 2; ++c)
#pragma unroll
    for (int i = 0; i < 32; i += 2) {
      const int col = 32 * c + i;
      float& t = top[i / 2 & 3];
      const float x = __uint_as_float(v[c][i]), y = __uint_as_float(v[c][i + 1]);
      if constexpr (kAll) {
        t = fmaxf(fmaxf(t, x), y);
      } else {
        if (col >= cb && col < ce) t = fmaxf(t, x);
        if (col + 1 >= cb && col + 1 < ce) t = fmaxf(t, y);
      }
    }
  return fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
}

// Stores p = 2^((x - m) sigma + kLift) of a row's scores x in fp16 over the first half of their columns; returns their
// sum.  kAll: every column, as 2^(x sigma + mneg), mneg = kLift - m sigma, whose rounding is 2^-11 at kFarScore; further
// on it would show, and pass the exponential's range at last, so those rows take the other form.
template <bool kAll>
__device__ __forceinline__ float row_exp(const uint32_t (&v)[2][32], uint32_t ts, float sigma, float m, float mneg, int cb,
                                         int ce) {
  const auto power = [&](uint32_t bits) {
    const float x = __uint_as_float(bits);
    return kAll ? ex2(fmaf(x, sigma, mneg)) : ex2(fmaf(x - m, sigma, kLift));
  };
  float part[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    uint32_t p[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      float x = power(v[c][2 * i]), y = power(v[c][2 * i + 1]);
      if constexpr (!kAll) {
        const int col = 32 * c + 2 * i;
        if (col < cb || col >= ce) x = 0.0f;
        if (col + 1 < cb || col + 1 >= ce) y = 0.0f;
      }
      part[2 * (i & 1)] += x;
      part[2 * (i & 1) + 1] += y;
      p[i] = half2_bits(x, y);
    }
    tmem_st16(ts + 16 * c, p);
  }
  return (part[0] + part[1]) + (part[2] + part[3]);
}

// Parts of rows for the join, of each block's 256 rows: D sums, and (log2 maximum, sum).
template <int G>
struct Parts {
  float* sums;  // [blocks][256][D]
  float2* ml;   // [blocks][256]
};

template <int G, bool kSplit>
__global__ void __launch_bounds__(kThreads, 1)
    attention_kv4_prompt(const __grid_constant__ Attn4 a, int min_rows, int sms, const Parts<G> parts) {
  using L = Layout<G>;
  constexpr int D = L::D;
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t raw_full[2][kRaw], raw_empty[2][kRaw], k_full[kBuf], k_empty[kBuf],
      v_full[kBuf], v_empty[kBuf], s_full[2][2], p_full[2][2], o_done[2][2], q_full[2], drained;
  __shared__ uint32_t tmem_slot;
  __shared__ int q_exp[kRows];  // of the power of two that a row of bf16 queries is scaled by
  const uint32_t sm = (smem_u32(smem_raw) + 1023u) & ~1023u;
  uint8_t* smp = smem_raw + (sm - smem_u32(smem_raw));
  const int tid = threadIdx.x, lane = tid & 31, warp = tid / 32;

  if (tid == 0) {
    for (int i = 0; i < 2 * kRaw; ++i) {
      mbar_init(smem_u32(&raw_full[0][i]), 1);
      mbar_init(smem_u32(&raw_empty[0][i]), 4);
    }
    for (int i = 0; i < kBuf; ++i) {
      mbar_init(smem_u32(&k_full[i]), 4);
      mbar_init(smem_u32(&k_empty[i]), 2);
      mbar_init(smem_u32(&v_full[i]), 4);
      mbar_init(smem_u32(&v_empty[i]), 2);
      mbar_init(smem_u32(&s_full[0][i]), 1);
      mbar_init(smem_u32(&p_full[0][i]), 128);
      mbar_init(smem_u32(&o_done[0][i]), 1);
    }
    mbar_init(smem_u32(&q_full[0]), 4);
    mbar_init(smem_u32(&q_full[1]), 4);
    mbar_init(smem_u32(&drained), 2);
    fence_mbar_init();
  }
  pdl_trigger();
  pdl_wait();
  if (blockIdx.x == 0)
    for (int b = tid; b < a.B; b += kThreads) {
      int f, n, l;
      if (!attn4_sequence(a, b, f, n, l)) report(kDevBadArg, kSiteSequence);
    }
  Job job;
  const int splits = kSplit ? splits_of(a, min_rows, sms, lane) : 1;
  if (!find_job(a, min_rows, splits, blockIdx.x, lane, job)) return;  // the same for every warp
  if (warp == kMmaWarp) {
    tmem_alloc(smem_u32(&tmem_slot), 512);
    tmem_relinquish();
  }

  // the keys of each row tile, in steps from the CTA's first
  const int row0 = job.tile * kRows;
  const auto pos_of = [&](int row) { return job.len - job.n + row / a.group; };
  const auto end_of = [&](int row) { return max(0, a.causal ? min(job.len, pos_of(row) + 1) : job.len); };
  const auto beg_of = [&](int row) { return attn4_oldest(a, pos_of(row)); };
  const int step0 = min(beg_of(row0), job.len) / kKeys;
  int steps[2];
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    const int last = min(row0 + 128 * t + 127, job.rows - 1);
    steps[t] = row0 + 128 * t < job.rows ? max(0, (end_of(last) + kKeys - 1) / kKeys - step0) : 0;
  }
  const int all = max(steps[0], steps[1]);
  const int j0 = (int)((int64_t)all * job.split / splits), j1 = (int)((int64_t)all * (job.split + 1) / splits);
#pragma unroll
  for (int t = 0; t < 2; ++t) steps[t] = max(0, min(steps[t], j1) - j0);
  const int total = max(steps[0], steps[1]);
  const int first_step = step0 + j0;
  const int lo = min(beg_of(row0), job.len);  // the oldest key that any row sees

  tc_fence_before();
  cta_barrier_all();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;
  const uint32_t tm_s = tmem, tm_o = tmem + 256;  // S: 2 x 64 columns a tile, in turn; O: D columns a tile

  // each group of four warps changes its registers at the head of its own branch
  if (warp < kSoftmaxWarp) {
    regs_down<kOtherRegs>();
    if (warp >= kLoadWarp) {
      // ---- packed codes and params: one warp for the keys' ring, one for the values' ---------
      const int ring = warp - kLoadWarp;
      const uint32_t base = sm + (ring ? L::values : L::keys), stage_bytes = ring ? L::kValueStage : L::kKeyStage;
      const int P = a.cache.page_size;
      const int piece = min(kKeys, P & -P), pieces = kKeys / piece;
      const int arr = lane / pieces, pc = lane % pieces;  // 0 codes, 1 params, 2 (keys' ring) the values' params
      const int arrays = ring ? 2 : 3;
      const uint32_t bytes = arr == 0 ? piece * (D / 2) : piece * (G * 4);
      const uint32_t dst_off = (arr == 0 ? 0 : L::kCodes + (arr - 1) * L::kParams) + pc * bytes;
      const uint32_t code_lanes = (1u << pieces) - 1;
      const uint32_t* src = arr == 0 ? (ring ? a.cache.codes[1] : a.cache.codes[0])
                                     : (ring || arr == 2 ? a.cache.params[1] : a.cache.params[0]);
      int issued = 0;
#pragma unroll 1
      for (int i = 0; i < total; ++i) {
        int page = -1, in_page = 0;
        const int t = first_step * kKeys + i * kKeys + pc * piece;
        if (arr < arrays && t < job.len) {
          const int pi = (int)kv4_page(a.cache, (uint32_t)t >> 4);
          in_page = t - pi * P;
          page = __ldg(a.table + (int64_t)job.b * a.table_ld + pi);
          if (page < 0 || page >= a.cache.pages) {
            report(kDevBadArg, kSitePage);
            page = -1;
          } else if (!dcheck(in_area(in_page, piece, P) && in_area(dst_off, bytes, stage_bytes) && (dst_off | bytes) % 16 == 0,
                             &g_status_prompt, kSiteCopy)) {
            page = -1;
          }
        }
        const int st = i % kRaw;
        if (!__all_sync(0xffffffffu, mbar_wait(smem_u32(&raw_empty[ring][st]), (i / kRaw & 1) ^ 1, &g_status_prompt, kSiteRawEmpty))) break;
        const uint32_t have = __ballot_sync(0xffffffffu, page >= 0);
        const uint32_t bar = smem_u32(&raw_full[ring][st]);
        if (lane == 0)
          mbar_arrive_expect_tx(bar, __popc(have & code_lanes) * (uint32_t)(piece * (D / 2)) +
                                         __popc(have & ~code_lanes) * (uint32_t)(piece * (G * 4)));
        __syncwarp();
        if (page >= 0) {
          const int64_t r = kv4_row(a.cache, page, job.h) + in_page;
          bulk_load(base + st * stage_bytes + dst_off, src + r * (arr == 0 ? D / 8 : G), bytes, bar);
        }
        issued = i + 1;
      }
      // no copy in flight outlives the CTA
      for (int i = max(0, issued - kRaw); i < issued; ++i)
        mbar_wait(smem_u32(&raw_full[ring][i % kRaw]), i / kRaw & 1, &g_status_prompt, kSiteDrain);
    } else {
      // ---- tensor cores, row tile `warp` ---------------------------------------------------------
      // The whole warp runs this with warp-uniform operands and one elected lane issues: from a branch of one lane the
      // operands go through vector registers and an MMA costs 175 cycles instead of 65.
      constexpr uint32_t kIdescS = idesc_f16_f32(128, kKeys), kIdescO = idesc_f16_f32(128, D);
      // descriptors of the operands' first blocks; a step along K or a block further only adds to the address field
      const uint64_t dq = sdesc_sw128(sm + L::q), dk = sdesc_sw128(sm + L::k), dv = sdesc_sw128(sm + L::v);
      const uint32_t um_s = __shfl_sync(0xffffffffu, tm_s, 0), um_o = __shfl_sync(0xffffffffu, tm_o, 0);
      const int t = __shfl_sync(0xffffffffu, warp, 0), mine = steps[t];
      const auto scores = [&](int i) {
        const uint64_t q = dq + (uint32_t)t * (L::kOperand >> 4), k = dk + (uint32_t)(i % kBuf) * (L::kStep >> 4);
        const uint32_t d = um_s + (i & 1) * 64 + t * 128;
        if (elect_one()) {
          mma_first(d, q, k, kIdescS);
#pragma unroll
          for (int n = 1; n < 4 * G; ++n)
            mma_next(d, q + (uint32_t)((n / 4 * L::kBlock + n % 4 * 32) >> 4),
                     k + (uint32_t)((n / 4 * (kKeys * 128) + n % 4 * 32) >> 4), kIdescS);
          mma_commit(smem_u32(&s_full[t][i & 1]));
          mma_commit(smem_u32(&k_empty[i % kBuf]));
        }
        __syncwarp();
      };
      const auto outputs = [&](int i) {
        const uint64_t v = dv + (uint32_t)(i % kBuf) * (L::kStep >> 4);
        const uint32_t d = um_o + t * D, p = um_s + (i & 1) * 64 + t * 128;
        if (elect_one()) {
          mma_f16_ts(d, p, v, kIdescO, i > 0);
#pragma unroll
          for (int n = 1; n < 4; ++n) mma_next_ts(d, p + n * 8, v + (uint32_t)(n * 32 >> 4), kIdescO);
          mma_commit(smem_u32(&o_done[t][i & 1]));
          mma_commit(smem_u32(&v_empty[i % kBuf]));
        }
        __syncwarp();
      };
      const auto wait = [&](uint64_t& bar, int parity, uint32_t site) {
        const bool ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(&bar), parity, &g_status_prompt, site));
        tc_fence_after();
        return ok;
      };
      // Scores run two steps ahead of the outputs, into the columns whose P the product before them has read (the
      // tensor cores work in order): a tile's next scores are there when its softmax comes to them.
      bool ok = mine == 0 || wait(q_full[t], 0, kSiteQ);
#pragma unroll 1
      for (int i = -2; i < mine && ok; ++i) {
        const int next = i + 2;
        if (i >= 0) {
          ok = wait(v_full[i % kBuf], i / kBuf & 1, kSiteVFull) && wait(p_full[t][i & 1], i >> 1 & 1, kSiteP);
          if (ok) outputs(i);
        }
        if (ok && next < mine) {
          ok = wait(k_full[next % kBuf], next / kBuf & 1, kSiteKFull);
          if (ok) scores(next);
        }
      }
      // the other tile's further steps want this one's part of their barriers (once the step's own phase has begun)
#pragma unroll 1
      for (int i = mine; i < total && ok; ++i) {
        ok = wait(k_full[i % kBuf], i / kBuf & 1, kSiteKFull) && wait(v_full[i % kBuf], i / kBuf & 1, kSiteVFull);
        if (ok && lane == 0) {
          mbar_arrive(smem_u32(&k_empty[i % kBuf]));
          mbar_arrive(smem_u32(&v_empty[i % kBuf]));
        }
      }
      if (elect_one()) mma_commit(smem_u32(&drained));
      __syncwarp();
      mbar_wait(smem_u32(&drained), 0, &g_status_prompt, kSiteDrain);
      __syncwarp();
    }
  } else if (warp >= kValueWarp) {
    regs_down<kDequantRegs>();
    // ---- values to fp16: a lane takes one word (8 channels) of 8 tokens and writes 8 tokens of 8 channels ----
    const int dt = tid - 32 * kValueWarp;
    if (a.dtype != QG_F16) {
      // The exponents of the rows' scales, while there are no values yet: a row's own, so that a NaN or a large query
      // does not cost the other rows digits.  (The softmax warps' own reduction took 6 to 13 % of the time of long
      // prompts: registers of their loop went to it.)
#pragma unroll 1
      for (int r = dt; r < kRows; r += 128) {
        const int row = row0 + r;
        uint32_t most = 0;  // of the magnitudes' bits
        if (row < job.rows) {
          const uint4* p = reinterpret_cast<const uint4*>(
              static_cast<const char*>(a.q) +
              2 * ((job.first + row / a.group) * a.q_st + (job.h * a.group + row % a.group) * a.q_sh));
#pragma unroll
          for (int k = 0; k < D / 8; ++k) {
            const uint4 x = __ldg(p + k);
            const auto larger = [](uint32_t w) { return max(w << 16 & 0x7FFF0000u, w & 0x7FFF0000u); };
            most = max(most, max(max(larger(x.x), larger(x.y)), max(larger(x.z), larger(x.w))));
          }
        }
        q_exp[r] = max(-120, min(100, 8 - ((int)(most >> 23) - 127)));
      }
      exponents_barrier();
    }
    const int jw = dt & 7, g = G == 2 ? dt >> 3 & 1 : 0, tg = dt >> (G == 2 ? 4 : 3);
    const int swap = tg & 1;  // odd groups read their pairs the other way round: no bank twice
    const uint32_t sel_lo = swap ? 0x1054u : 0x5410u, sel_hi = swap ? 0x3276u : 0x7632u;
#pragma unroll 1
    for (int i = 0; i < total; ++i) {
      const int buf = i % kBuf, st = i % kRaw;
      bool ok = mbar_wait(smem_u32(&v_empty[buf]), (i / kBuf & 1) ^ 1, &g_status_prompt, kSiteVEmpty);
      if (ok) ok = mbar_wait(smem_u32(&raw_full[1][st]), i / kRaw & 1, &g_status_prompt, kSiteRawFull);
      if (!__all_sync(0xffffffffu, ok)) break;
      const uint8_t* vc = smp + L::values + st * L::kValueStage;
      const uint8_t* vp = vc + L::kCodes;
      const int t0 = (first_step + i) * kKeys;
      const bool odd = any_odd<kKeys * G>(vp, lane) || t0 < lo || t0 + kKeys > job.len;
      if (G == 2 || dt < 64) {
        uint32_t pw[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) pw[k] = *reinterpret_cast<const uint32_t*>(vp + ((tg * 8 + k) * G + g) * 4);
        if (odd) {  // tokens that no row sees: zero
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const int t = t0 + tg * 8 + k;
            if (t < lo || t >= job.len) pw[k] = 0u;
          }
        }
        uint32_t out[8][4];  // channel, token pair
#pragma unroll
        for (int p = 0; p < 4; ++p) {
          const uint8_t* src = vc + (tg * 8 + 2 * p) * (D / 2) + (jw * G + g) * 4;
          const uint32_t x = *reinterpret_cast<const uint32_t*>(src + swap * (D / 2));
          const uint32_t y = *reinterpret_cast<const uint32_t*>(src + (swap ^ 1) * (D / 2));
          const uint32_t s2 = __byte_perm(pw[2 * p], pw[2 * p + 1], 0x5410);
          const uint32_t o2 = __byte_perm(pw[2 * p], pw[2 * p + 1], 0x7632);
#pragma unroll
          for (int hh = 0; hh < 2; ++hh) {  // nibbles 0..3, 4..7
            uint32_t c[4];
            codes_f16(__byte_perm(x, y, hh ? sel_hi : sel_lo), c);
#pragma unroll
            for (int m = 0; m < 4; ++m) out[4 * hh + m][p] = h2_fma(c[m], s2, o2);
          }
        }
        if (odd) {  // finite (hidden tokens meet p = 0); a visible token's NaN comes through its key
#pragma unroll
          for (int c = 0; c < 8; ++c)
#pragma unroll
            for (int p = 0; p < 4; ++p) out[c][p] = h2_finite(out[c][p]);
        }
        // row 64 g + 8 i + jw, keys 8 tg ..: chunk tg
        const uint32_t vrow = sm + L::v + buf * L::kStep + (64 * g + jw) * 128 + ((tg ^ jw) << 4);
#pragma unroll
        for (int i2 = 0; i2 < 8; ++i2) sts128(vrow + i2 * 8 * 128, out[i2][0], out[i2][1], out[i2][2], out[i2][3]);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(smem_u32(&raw_empty[1][st]));
        mbar_arrive(smem_u32(&v_full[buf]));
      }
    }
  } else if (warp >= kKeyWarp) {
    regs_down<kDequantRegs>();
    // ---- keys to fp16: a lane takes 4 words (32 channels) of a token ----------------------------
    const int dt = tid - 32 * kKeyWarp;
    constexpr int kParts = D / 32;  // lanes per token
#pragma unroll 1
    for (int i = 0; i < total; ++i) {
      const int buf = i % kBuf, st = i % kRaw;
      bool ok = mbar_wait(smem_u32(&k_empty[buf]), (i / kBuf & 1) ^ 1, &g_status_prompt, kSiteKEmpty);
      if (ok) ok = mbar_wait(smem_u32(&raw_full[0][st]), i / kRaw & 1, &g_status_prompt, kSiteRawFull);
      if (!__all_sync(0xffffffffu, ok)) break;
      const uint8_t* kc = smp + L::keys + st * L::kKeyStage;
      const uint8_t *kp = kc + L::kCodes, *vp = kp + L::kParams;
      const bool odd = any_odd<2 * kKeys * G>(kp, lane);  // the values' params lie behind the keys'
#pragma unroll
      for (int it = 0; it < kParts / 2; ++it) {
        const int item = dt + 128 * it, part = item % kParts, tok = item / kParts;
        uint32_t kpw[G], out[4][4];
#pragma unroll
        for (int g = 0; g < G; ++g) kpw[g] = *reinterpret_cast<const uint32_t*>(kp + (tok * G + g) * 4);
        const uint4 words = *reinterpret_cast<const uint4*>(kc + tok * (D / 2) + part * 16);
        const uint32_t* w = &words.x;
        uint32_t s2[G], o2[G];
#pragma unroll
        for (int g = 0; g < G; ++g) {
          s2[g] = __byte_perm(kpw[g], 0, 0x1010);
          o2[g] = __byte_perm(kpw[g], 0, 0x3232);
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          uint32_t c[4];
          codes_f16(w[k], c);
#pragma unroll
          for (int m = 0; m < 4; ++m) out[k][m] = h2_fma(c[m], s2[k % G], o2[k % G]);
        }
        if (odd) {
          // A token with params that are not finite gets a NaN key: every row that sees it becomes NaN, none else
          // (its value is taken finite).  Large keys are held to the type.
          bool bad = false;
#pragma unroll
          for (int g = 0; g < G; ++g)
            bad |= not_finite(kpw[g]) || not_finite(*reinterpret_cast<const uint32_t*>(vp + (tok * G + g) * 4));
#pragma unroll
          for (int k = 0; k < 4; ++k)
#pragma unroll
            for (int m = 0; m < 4; ++m) out[k][m] = bad ? 0x7FFF7FFFu : h2_finite(out[k][m]);
        }
        // word k of the lane is word [j, g] of the token: index part * 4 + k = j G + g
        const uint32_t krow = sm + L::k + buf * L::kStep + tok * 128;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int jw = (part * 4 + k) / G;
          sts128(krow + (k % G) * (kKeys * 128) + ((jw ^ (tok & 7)) << 4), out[k][0], out[k][1], out[k][2], out[k][3]);
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(smem_u32(&raw_empty[0][st]));
        mbar_arrive(smem_u32(&k_full[buf]));
      }
    }
  } else {
    regs_up<kSoftmaxRegs>();
    // ---- softmax, one thread per row ------------------------------------------
    // Rows move 16 bytes a lane, kLpr lanes a row; a lane knows the place of its own row, whose softmax it takes.
    constexpr int kLpr = D / 8, kRpi = 32 / kLpr;
    const int tile = (warp - kSoftmaxWarp) / 4 & 1, wrow = (warp & 3) * 32;  // the warp's rows in its tile
    const int row = row0 + tile * 128 + wrow + lane;
    const bool valid = row < job.rows;
    const int t_row = job.first + row / a.group, hq = job.h * a.group + row % a.group;
    const int piece = lane % kLpr, sub = lane / kLpr;
    uint4 qv[kLpr];
    {
      const int64_t mine_at = valid ? 2 * (t_row * a.q_st + hq * a.q_sh) : -1;
#pragma unroll
      for (int it = 0; it < kLpr; ++it) {
        const int64_t at = __shfl_sync(0xffffffffu, mine_at, it * kRpi + sub);
        qv[it] = at < 0 ? make_uint4(0u, 0u, 0u, 0u)
                        : __ldg(reinterpret_cast<const uint4*>(static_cast<const char*>(a.q) + at + 16 * piece));
      }
    }
    const uint32_t place = sm + L::q + tile * L::kOperand + (piece / 8) * L::kBlock;  // of the lane's 16 bytes in row 0
    const auto in_row = [&](int r) { return place + (wrow + r) * 128 + (((piece & 7) ^ (r & 7)) << 4); };
    // queries to fp16: as they are, or (bf16) scaled by the power of two that brings the row's largest near 2^8
    float sigma = a.scale * 1.44269504088896f;
    if (a.dtype == QG_F16) {
#pragma unroll
      for (int it = 0; it < kLpr; ++it)
        sts128(in_row(it * kRpi + sub), __byte_perm(qv[it].x, qv[it].z, 0x5410), __byte_perm(qv[it].x, qv[it].z, 0x7632),
               __byte_perm(qv[it].y, qv[it].w, 0x5410), __byte_perm(qv[it].y, qv[it].w, 0x7632));
    } else {
      exponents_barrier();  // they are there
      sigma *= __uint_as_float((uint32_t)(127 - q_exp[tile * 128 + wrow + lane]) << 23);
#pragma unroll
      for (int it = 0; it < kLpr; ++it) {
        const uint32_t* w = &qv[it].x;
        const float up = __uint_as_float((uint32_t)(127 + q_exp[tile * 128 + wrow + it * kRpi + sub]) << 23);
        const auto pair = [&](int i, int k) {  // values i and k
          const float x = __uint_as_float(i & 1 ? w[i / 2] & 0xffff0000u : w[i / 2] << 16);
          const float y = __uint_as_float(k & 1 ? w[k / 2] & 0xffff0000u : w[k / 2] << 16);
          return half2_bits(x * up, y * up);
        };
        sts128(in_row(it * kRpi + sub), pair(0, 4), pair(1, 5), pair(2, 6), pair(3, 7));
      }
    }
    sigma = fminf(sigma, 0x1p87f);  // scores, 2^39 at most, stay in binary32: by then the best key has all of the weight
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(&q_full[tile]));
    const int mine = steps[tile];
    const uint32_t lanes = (uint32_t)(warp & 3) << 21;  // tensor-memory lane 32 (warp % 4)
    const uint32_t to = tm_o + tile * D + lanes;
    const int last_row = min(row0 + 128 * tile + 127, job.rows - 1);
    const int r = min(row, last_row);  // rows behind the last: zero queries with its mask
    const int end = end_of(r), beg = beg_of(r);
    const int min_end = end_of(row0 + 128 * tile), max_beg = beg_of(last_row);
    float m = -INFINITY, mneg = 0.0f, l = 0.0f;  // the maximum taken against, kLift - m sigma, the sum of p 2^kLift
    bool ok = true, far_scores = false;  // a row of the warp has a maximum beyond kFarScore
#pragma unroll 1
    for (int j = 0; j < mine; ++j) {
      const uint32_t ts = tm_s + tile * 128 + (j & 1) * 64 + lanes;
      ok = mbar_wait(smem_u32(&s_full[tile][j & 1]), j >> 1 & 1, &g_status_prompt, kSiteS);
      if (!__all_sync(0xffffffffu, ok)) break;
      tc_fence_after();
      const int t0 = (first_step + j) * kKeys;
      const bool full = t0 >= max_beg && t0 + kKeys <= min_end;
      const int cb = beg - t0, ce = end - t0;  // the visible columns [cb, ce)
      uint32_t v[2][32];
      tmem_ld32(ts, v[0]);
      tmem_ld32(ts + 32, v[1]);
      tmem_ld_wait();
      const float top = full ? row_max<true>(v, cb, ce) : row_max<false>(v, cb, ce);
      const bool far = top > -INFINITY && (m == -INFINITY || (top - m) * sigma > kAhead);
      if (__any_sync(0xffffffffu, far)) {
        const float mn = fmaxf(m, top);
        const float corr = m == -INFINITY ? 0.0f : ex2((m - mn) * sigma);
        m = mn;
        mneg = m == -INFINITY ? 0.0f : fmaf(-m, sigma, kLift);
        far_scores = __any_sync(0xffffffffu, fabsf(mneg) > kFarScore);
        l *= corr;
        if (j > 0) {
          // (of that barrier's phases all but this one are done: step j - 3's product came before step j - 1's scores)
          ok = mbar_wait(smem_u32(&o_done[tile][(j - 1) & 1]), (j - 1) >> 1 & 1, &g_status_prompt, kSiteO);
          if (!__all_sync(0xffffffffu, ok)) break;
          tc_fence_after();
#pragma unroll
          for (int c = 0; c < D / 16; ++c) {
            uint32_t u[16];
            tmem_ld16(to + 16 * c, u);
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 16; ++i) u[i] = __float_as_uint(__uint_as_float(u[i]) * corr);
            tmem_st16(to + 16 * c, u);
          }
        }
      }
      l += full && !far_scores ? row_exp<true>(v, ts, sigma, 0.0f, mneg, cb, ce)
                               : row_exp<false>(v, ts, sigma, m == -INFINITY ? 0.0f : m, 0.0f, cb, ce);
      tmem_st_wait();
      tc_fence_before();
      mbar_arrive(smem_u32(&p_full[tile][j & 1]));
    }
    // the output row
    for (int j = max(0, mine - 2); j < mine && ok; ++j)
      ok = mbar_wait(smem_u32(&o_done[tile][j & 1]), j >> 1 & 1, &g_status_prompt, kSiteO);
    ok = __all_sync(0xffffffffu, ok);
    tc_fence_after();
    const int64_t flat = (int64_t)blockIdx.x * kRows + tile * 128 + wrow + lane;  // of the parts
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    const uint32_t my_row = sm + L::q + tile * L::kOperand + (wrow + lane) * 128;  // the queries have been read
#pragma unroll
    for (int g = 0; g < G; ++g) {
      float v[64];
      if (mine > 0) {
        uint32_t u[32];
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {
          tmem_ld32(to + 64 * g + 32 * hh, u);
          tmem_ld_wait();
#pragma unroll
          for (int i = 0; i < 32; ++i) v[32 * hh + i] = __uint_as_float(u[i]);
        }
      }
      if (mine == 0 || l == 0.0f) {
#pragma unroll
        for (int i = 0; i < 64; ++i) v[i] = 0.0f;
      }
      // column 8 i + jw is channel 8 jw + i
      if (splits == 1) {
#pragma unroll
        for (int jw = 0; jw < 8; ++jw) {
          uint32_t b[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float x = v[16 * i + jw] * inv, y = v[16 * i + 8 + jw] * inv;
            if (a.dtype == QG_F16) {
              b[i] = half2_bits(x, y);
            } else {
              __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
              b[i] = *reinterpret_cast<uint32_t*>(&h);
            }
          }
          sts128(my_row + g * L::kBlock + ((jw ^ (lane & 7)) << 4), b[0], b[1], b[2], b[3]);
        }
      } else if (valid && ok) {
        float* p = parts.sums + flat * D + 64 * g;
#pragma unroll
        for (int jw = 0; jw < 8; ++jw) {
          *reinterpret_cast<float4*>(p + 8 * jw) = make_float4(v[jw], v[8 + jw], v[16 + jw], v[24 + jw]);
          *reinterpret_cast<float4*>(p + 8 * jw + 4) = make_float4(v[32 + jw], v[40 + jw], v[48 + jw], v[56 + jw]);
        }
      }
    }
    if (splits == 1) {
      __syncwarp();
      const int64_t mine_at = valid && ok ? 2 * (t_row * a.o_st + hq * a.o_sh) : -1;
#pragma unroll
      for (int it = 0; it < kLpr; ++it) {
        const int64_t at = __shfl_sync(0xffffffffu, mine_at, it * kRpi + sub);
        uint4 o;
        asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
                     : "=r"(o.x), "=r"(o.y), "=r"(o.z), "=r"(o.w)
                     : "r"(in_row(it * kRpi + sub)));
        if (at >= 0) *reinterpret_cast<uint4*>(static_cast<char*>(a.out) + at + 16 * piece) = o;
      }
    }
    if (valid && ok) {
      const float lg = l == 0.0f ? -INFINITY : m * sigma - kLift;  // log2 of what p was taken against
      if (splits > 1) parts.ml[flat] = make_float2(lg, l);
      else if (a.lse) a.lse[(int64_t)t_row * a.heads_q + hq] = l == 0.0f ? -INFINITY : (lg + log2f(l)) * 0.69314718056f;
    }
    tc_fence_before();
  }
  cta_barrier_all();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Joins the splits' parts: block (tile, head; 16 rows), a warp per row.
constexpr int kJoinRows = 16;
template <int G>
__global__ void __launch_bounds__(256)
    attention_kv4_prompt_join(const __grid_constant__ Attn4 a, int min_rows, int sms, const Parts<G> parts) {
  constexpr int D = 64 * G;
  pdl_trigger();
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
  Job job;
  const int splits = splits_of(a, min_rows, sms, lane);
  if (splits == 1 || !find_job(a, min_rows, 1, blockIdx.x, lane, job)) return;
  const int64_t stride = (int64_t)a.cache.heads * kRows;  // a split further
  const int64_t from = ((int64_t)(blockIdx.x / a.cache.heads * splits) * a.cache.heads + job.h) * kRows;
#pragma unroll 1
  for (int r = blockIdx.y * kJoinRows + warp; r < min((int)(blockIdx.y + 1) * kJoinRows, job.rows - job.tile * kRows); r += 8) {
    float v[D / 32], top, l;
    add_parts<D>([&](int i) { return parts.sums + (from + r + i * stride) * D; },
                 [&](int i) { return parts.ml + from + r + i * stride; }, splits, lane, top, l, v);
    write_row<D>(a, job.first, job.h, job.tile * kRows + r, lane, top, l, v);
  }
}

// Row tiles of a call (an upper bound where the sequences' row counts are on the device)
int64_t row_tiles(int64_t B, int64_t T, int64_t group, bool ragged) {
  return ragged ? T * group / kRows + B : B * ((T / B * group + kRows - 1) / kRows);
}

// Rows (query tokens x head group) that the decode kernel takes, in tiles of 8; 0: none.  A ragged call gives it
// the sequences of 8 rows at most, or of 16 where one token has more than 8 or the mean sequence has 9 to 16 (drafts;
// 64 sequences of 4096..8192 tokens, 32/8 heads of 128, 60 of them with 3 new tokens: 180 us, 457 with the prompt kernel for
// these; but one of them with 3: 170, 144 with the prompt kernel for it).
int decode_tiles(int64_t B, int64_t T, int64_t group, bool ragged) {
  int64_t rows = T / B * group;
  if (ragged) rows = T * group > 8 * B && T * group <= 16 * B ? 16 : group;
  return rows <= 8 ? 1 : rows <= 16 ? 2 : 0;
}

// Blocks of a call, and those that leave parts (0: every tile's keys are one share, and the kernel without parts takes
// them, 13 us less for 2 x 4096 tokens of 32 heads).  The device counts a ragged call's tiles, but the query
// tokens that its sequences share make a least number of them, with which nothing is split.
struct Blocks {
  int64_t all, parts;
};
Blocks blocks_of(int64_t B, int64_t T, int64_t group, int64_t heads, bool ragged, int nt) {
  const int64_t items = row_tiles(B, T, group, ragged) * heads;
  if (ragged) {
    const int64_t rows = T * group - B * 8 * nt, least = rows > 0 ? (rows + kRows - 1) / kRows * heads : 0;
    if (2 * least > sm_count()) return {items, 0};
    return {std::max<int64_t>(items, sm_count()), sm_count()};  // tiles x heads x splits: the SMs at most
  }
  const int splits = key_splits(items, 1, sm_count());
  return {items * splits, splits > 1 ? items * splits : 0};
}

template <int G>
Parts<G> parts_of(int64_t blocks, void* workspace) {
  Parts<G> p;
  p.sums = static_cast<float*>(workspace);
  p.ml = reinterpret_cast<float2*>(p.sums + blocks * kRows * 64 * G);
  return p;
}

template <int G, bool kSplit>
qg_status launch(const Attn4& a, int min_rows, const Blocks& n, void* workspace, cudaStream_t s) {
  constexpr int kSmem = Layout<G>::bytes + 1024;
  static PerDeviceOnce once;
  const qg_status st = once.run([](int) {
    // the warps' register shares are drawn on the block's own: fewer at launch would wait for ever
    cudaFuncAttributes f;
    const qg_status q = check_cuda(cudaFuncGetAttributes(&f, attention_kv4_prompt<G, kSplit>), "attention_kv4 attributes");
    if (q != QG_OK) return q;
    if (f.numRegs < kLaunchRegs) return fail(QG_ERR_UNSUPPORTED, "attention_kv4: built with %d registers a thread, %d needed", f.numRegs, kLaunchRegs);
    return check_cuda(cudaFuncSetAttribute(attention_kv4_prompt<G, kSplit>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem),
                      "attention_kv4 shared memory");
  });
  if (st != QG_OK) return st;
  if (n.all >= ((int64_t)1 << 31)) return fail(QG_ERR_UNSUPPORTED, "attention_kv4: too many row tiles");
  LaunchCfg lc((unsigned)n.all, kThreads, kSmem, s);
  return check_cuda(cudaLaunchKernelEx(&lc.cfg, attention_kv4_prompt<G, kSplit>, a, min_rows, sm_count(), parts_of<G>(n.parts, workspace)),
                    "attention_kv4 prompt launch");
}

template <int G>
qg_status launch_join(const Attn4& a, int min_rows, const Blocks& n, void* workspace, cudaStream_t s) {
  LaunchCfg lc((unsigned)(n.parts / 2), 256, 0, s);  // two splits or more each
  lc.cfg.gridDim.y = kRows / kJoinRows;
  return check_cuda(cudaLaunchKernelEx(&lc.cfg, attention_kv4_prompt_join<G>, a, min_rows, sm_count(), parts_of<G>(n.parts, workspace)),
                    "attention_kv4 prompt join launch");
}

size_t round256(size_t n) { return (n + 255) / 256 * 256; }

}  // namespace

size_t attention_kv4_workspace(int64_t B, int64_t T, int64_t heads_q, int64_t heads, int64_t dim, bool ragged) {
  const int64_t group = heads_q / heads;
  const int nt = decode_tiles(B, T, group, ragged);
  size_t bytes = nt ? round256(attention_kv4_decode_workspace(dim, nt)) : 0;
  if (!nt || ragged) {
    bytes += (size_t)blocks_of(B, T, group, heads, ragged, nt).parts * kRows * (dim + 2) * sizeof(float);
  }
  return bytes;
}

// Single tokens and drafts go to the decode kernel, longer ones here; a ragged call launches both and each takes its
// sequences, the prompts first.
qg_status launch_attention_kv4(const Attn4& a, void* workspace, cudaStream_t s) {
  const int nt = decode_tiles(a.B, a.T, a.group, a.q_starts != nullptr);
  const bool prompts = !nt || a.q_starts;
  const Blocks n = blocks_of(a.B, a.T, a.group, a.cache.heads, a.q_starts != nullptr, nt);
  const int min_rows = 8 * nt + 1;
  void* const mine = static_cast<char*>(workspace) + (nt ? round256(attention_kv4_decode_workspace(a.cache.dim, nt)) : 0);
  qg_status st = QG_OK;
  if (prompts && a.cache.dim == 64)
    st = n.parts ? launch<1, true>(a, min_rows, n, mine, s) : launch<1, false>(a, min_rows, n, mine, s);
  else if (prompts)
    st = n.parts ? launch<2, true>(a, min_rows, n, mine, s) : launch<2, false>(a, min_rows, n, mine, s);
  if (st == QG_OK && nt) st = launch_attention_kv4_decode(a, nt, workspace, s);
  if (st == QG_OK && prompts && n.parts)
    st = a.cache.dim == 64 ? launch_join<1>(a, min_rows, n, mine, s) : launch_join<2>(a, min_rows, n, mine, s);
  if (st == QG_OK && nt) st = launch_attention_kv4_decode_join(a, nt, workspace, s);
  return st;
}

}  // namespace qg
