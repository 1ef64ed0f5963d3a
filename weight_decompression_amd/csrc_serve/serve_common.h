// Shared by the serving kernels (paged cache, attention, drafts): the cache's block layout,
// the batch description as kernels see it, and small conversions.  gfx950 only.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "llvq.h"

namespace serve {

using bf16x2 = __bf16 __attribute__((ext_vector_type(2)));
using bf16x8 = __bf16 __attribute__((ext_vector_type(8)));
using f32x2 = float __attribute__((ext_vector_type(2)));
using f32x4 = float __attribute__((ext_vector_type(4)));
using f32x16 = float __attribute__((ext_vector_type(16)));
using u32x2 = uint32_t __attribute__((ext_vector_type(2)));
using u32x4 = uint32_t __attribute__((ext_vector_type(4)));
using s16x4 = short __attribute__((ext_vector_type(4)));

constexpr int kGroup = 32;  // channels that share a scale
constexpr int kWave = 64;
constexpr int kMaxLen = 1 << 30;  // tokens of a sequence, and of a window

// Bytes of one token's codes of one head.
__host__ __device__ constexpr int code_bytes(int kind, int dim) {
  return kind == LLVQ_KV_BF16 ? 2 * dim : kind == LLVQ_KV_FP8 ? dim : dim / 2;
}

// The last scale byte that stands for a power of two (e = 119 and 125: the largest codes, 448 and 6, times 2^e stay
// below 2^128).  Those past it stand for NaN; a write leaves none of them but 255.
__host__ __device__ constexpr int last_scale(int kind) { return kind == LLVQ_KV_FP8 ? 246 : 252; }

// n / d for 0 <= n < 2^31 as (n * mul) >> shift: with s = ceil(log2 d) and mul =
// ceil(2^(31+s) / d) < 2^32, mul * d exceeds 2^(31+s) by less than d <= 2^s, so the quotient
// is exact.
struct Divider {
  uint32_t mul, shift, by;
};
inline Divider make_divider(uint32_t d) {
  uint32_t s = 0;
  while ((1ull << s) < d) ++s;
  return {(uint32_t)(((1ull << (31 + s)) + d - 1) / d), 31 + s, d};
}
__device__ __forceinline__ uint32_t divide(uint32_t n, const Divider& d) {
  return (uint32_t)(((uint64_t)n * d.mul) >> d.shift);
}

// A paged cache and a batch of sequences over it.
struct Cache {
  uint8_t* pool;
  const int32_t* starts;  // [batch + 1]
  const int32_t* lens;    // [batch]
  const int32_t* table;   // [batch][max_pages]
  int64_t block;          // bytes of one (page, head)
  Divider page;           // tokens of a page
  int32_t heads, dim, pages, batch, max_pages, tokens;
  int32_t row, groups;                   // code bytes and scale bytes of one token
  int32_t v_off, ks_off, vs_off;         // from the block's start
};

// One sequence, with what the arrays say cut to what the batch and its table hold.
struct Seq {
  int32_t first, n, len;  // first row of the new tokens, their number, the cached tokens
  bool bad;
};
__device__ __forceinline__ Seq sequence(const Cache& c, int b) {
  const int32_t s0 = c.starts[b], s1 = c.starts[b + 1], len = c.lens[b];
  const int64_t cap = (int64_t)c.max_pages * c.page.by;
  const int32_t most = (int32_t)(cap < kMaxLen ? cap : kMaxLen);
  Seq s;
  s.first = min(max(s0, 0), c.tokens);
  s.n = min(max(s1, s.first), c.tokens) - s.first;
  s.len = min(max(len, 0), most);
  s.bad = s0 != s.first || s1 != s.first + s.n || len != s.len;
  return s;
}

// Offset of a token's block in the pool, or -1 for a page number outside the pool.
__device__ __forceinline__ int64_t block_of(const Cache& c, int b, uint32_t page, int head) {
  const int32_t id = c.table[(int64_t)b * c.max_pages + page];
  if (id < 0 || id >= c.pages) return -1;
  return ((int64_t)id * c.heads + head) * c.block;
}

__device__ __forceinline__ float bf16_f32(uint16_t b) { return __uint_as_float((uint32_t)b << 16); }
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  const f32x2 v = {a, b};
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2));
}

// The sequence that holds new token t: the number of sequences that end at or before it.
// Every lane of the wave has the same t; 64 ends are compared at a time.
__device__ __forceinline__ int sequence_of(const Cache& c, int t) {
  const int lane = threadIdx.x & 63;
  int n = 0;
  for (int base = 0; base < c.batch; base += kWave) {
    const bool in = base + lane < c.batch;
    const int32_t end = in ? c.starts[base + lane + 1] : 0x7fffffff;
    n += __popcll(__ballot(end <= t));
  }
  return n;
}

}  // namespace serve
