// qg_kv4.cuh -- the paged 4-bit key/value cache shared by its writer, reader
// and the attention kernels.
//
// A page holds `page_size` tokens of every KV head; for each (page, head) the
// codes of a token are D/8 words of 8 codes and its params D/64 pairs:
//   codes  [pages, heads, page_size, 8, D/64] words: word [j, g] holds channels
//          64 g + 8 j .. + 7, channel i of them in bits 4 i
//   params [pages, heads, page_size, D/64] (scale, offset) fp16 pairs
//   value = scale * code + offset
// One (page, head) is one contiguous block of each array, a multiple of 16
// bytes, so it moves by plain bulk copies; the words of one j for all groups
// lie side by side, so the lane that owns 8 channels of each group reads them
// with one load.
#pragma once

#include <stdint.h>

#include "../../include/qg.h"

namespace qg {

struct KV4 {
  uint32_t* codes[2];   // keys, values
  uint32_t* params[2];  // fp16 (scale, offset) in one word
  int64_t pages;
  int heads, page_size, dim;
  // floor(n / (page_size / 16)) = n * magic >> shift for n < 2^31: magic = ceil(2^shift / k), 2^(shift - 32) <= k,
  // so n * (magic - 2^shift / k) < 2^31 < 2^shift / k and n * magic < 2^64
  uint64_t page_magic;
  int page_shift;
};

// The page of a token position below 2^35 (page_size is a multiple of 16)
__host__ __device__ __forceinline__ uint32_t kv4_page(const KV4& c, uint32_t sixteenths) {
  return (uint32_t)(sixteenths * c.page_magic >> c.page_shift);
}

// First token row of (page, head)
__host__ __device__ __forceinline__ int64_t kv4_row(const KV4& c, int64_t page, int head) {
  return (page * c.heads + head) * (int64_t)c.page_size;
}

// Attention over the cache: T query tokens of B sequences, row t of q is token
// t of all sequences back to back.
struct Attn4 {
  KV4 cache;
  const void* q;        // [T, heads_q, dim] of `dtype`, strides in elements
  void* out;
  int64_t q_st, q_sh, o_st, o_sh;
  float* lse;           // [T, heads_q] or NULL
  const int32_t* table; // [B, max_pages], row stride table_ld
  int64_t table_ld;
  const int32_t* seq_lens;  // [B]
  const int32_t* q_starts;  // [B + 1], or NULL: n_uniform tokens per sequence
  int n_uniform;
  int B, T, heads_q, group;  // group = heads_q / heads
  int max_pages;
  float scale;
  int causal;
  int window;  // 0: none
  int dtype;
};

#ifdef __CUDACC__
// A sequence's query tokens [first, first + n) and its length, held to what
// the arguments cover; false if the device data had to be cut.
__device__ __forceinline__ bool attn4_sequence(const Attn4& a, int b, int& first, int& n, int& len) {
  bool ok = true;
  if (a.q_starts) {
    const int s0 = a.q_starts[b], s1 = a.q_starts[b + 1];
    ok = s0 >= 0 && s1 >= s0 && s1 <= a.T;
    first = s0;
    n = ok ? s1 - s0 : 0;
  } else {
    first = b * a.n_uniform;
    n = a.n_uniform;
  }
  len = a.seq_lens[b];
  const int64_t room = (int64_t)a.max_pages * a.cache.page_size;
  if (len < 0 || len > room) {
    ok = false;
    len = len < 0 ? 0 : (int)room;
  }
  return ok;
}

// The oldest key that a query at `pos` sees.  (It may stand before the sequence, where pos - window + 1 can leave 32
// bits: any such place gives 0.)
__device__ __forceinline__ int attn4_oldest(const Attn4& a, int pos) {
  return a.window > 0 ? max(0, max(pos, -1) - a.window + 1) : 0;
}
#endif

}  // namespace qg
