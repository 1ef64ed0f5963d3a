// The move of the tokens that stay to the front of their sequence: place first + i takes what lies at first + keep[i],
// keep ascending, in place and for each key head by its own list.
//
// What moves is read once and written once; HBM bounds it for long lists, the launch for short ones.  A token's parts (key and
// value codes, their scale bytes, its weight) never meet, so a workgroup has one part of a (sequence, key head), of the
// codes 64 to 256 bytes of each row, and takes the list in order, a batch of entries at a time: all of a batch is read, then, after
// a barrier, written.  That is enough for moves in place: keep[i] >= i, so what a batch writes (its own i) lies before
// anything that later batches read (at or past their own, larger i), and what earlier batches read is past the barrier.  The
// loads of the next batch are under way while a batch is written.  Where entries lie is worked out for 1024 at a time, into LDS:
// left to each batch, list, page and codes are three loads that wait for each other.
//
// Measured: 8192 of up to 32768 tokens of 8 sequences and 8 heads of 128 channels in bf16, weights too: 130 us (a call 133), 4.1 TB/s read and
// written, where a large copy reaches 5.1; in e4m3 71 (3.9), in e2m1 56 (2.6): one workgroup has all scale bytes of a (sequence,
// key head), so 8192 of one sequence take 36 us in bf16 and 50 in e4m3 and e2m1.  2048 of 2304 of one sequence 11 us (e4m3 15);
// accepted paths of 16 trees 4.3 us (e4m3 6.4), a launch and the chain of loads.
#pragma once

#include "serve_common.h"

namespace serve {

struct KeepArgs {
  Cache c;
  float* weights;         // [pages][heads][page] or null
  const int32_t* keep;    // [batch][lists][width]
  const int32_t* counts;  // [batch] or null
  int32_t lists, width;   // lists: 1, or one for each key head
  bool from_new;          // entries count from the first new token, not from the first of all
  int32_t* err;
  int32_t side, slices;   // 16-byte chunks of a slice, and slices of a row of codes
  int32_t parts;          // workgroups a (sequence, key head): slices of keys, slices of values, scales, weights
};

constexpr int kKeepThreads = 1024, kKeepAhead = 4, kKeepList = 1024;

// The list of a (sequence, key head), and where its entries lie: (page * heads + head) and slot, from and to (-1: nothing moves).
struct Moves {
  const int32_t* keep;
  const int32_t* table;
  int count, first, len, head;
};
using Entry = int __attribute__((ext_vector_type(4)));
__device__ __forceinline__ Entry entry_of(const Cache& c, const Moves& m, int i, bool* bad) {
  const Entry none = {-1, 0, 0, 0};
  if (i >= m.count) return none;
  const int k = m.keep[i], last = i > 0 ? m.keep[i - 1] : -1;
  if (k == i || k == -1) return none;
  if (k < i || (i > 0 && k <= last) || k >= m.len - m.first) {
    *bad = true;
    return none;
  }
  const uint32_t src = (uint32_t)(m.first + k), dst = (uint32_t)(m.first + i);
  const uint32_t sp = divide(src, c.page), dp = divide(dst, c.page);
  const int32_t s = m.table[sp], d = m.table[dp];
  if (s < 0 || s >= c.pages || d < 0 || d >= c.pages) {
    *bad = true;
    return none;
  }
  return Entry{s, (int)(src - sp * c.page.by), d, (int)(dst - dp * c.page.by)};
}

// Moves `per` elements of T of every entry's row, `side` threads an entry: element e of a token lies at base + block * stride +
// slot * row + e.  Returns whether an entry was bad.
template <typename T, int AHEAD>
__device__ __forceinline__ bool move_part(const Cache& c, const Moves& m, Entry* list, uint8_t* base, int64_t stride, int row, int per,
                                          int side) {
  const int tid = threadIdx.x;
  const int entry = tid / side, lane = tid % side, entries = (int)blockDim.x / side, step = entries * AHEAD;
  bool bad = false;
  for (int i0 = 0; i0 < m.count; i0 += kKeepList) {
    const int n = min(m.count - i0, kKeepList);
    __syncthreads();  // (the list before has been used)
    for (int i = tid; i < n; i += (int)blockDim.x) list[i] = entry_of(c, m, i0 + i, &bad);
    __syncthreads();
    for (int e0 = 0; e0 < per; e0 += side) {
      const int e = e0 + lane;
      T data[2][AHEAD];
      int64_t to[2][AHEAD];
      auto load = [&](int round, int at) {
#pragma unroll
        for (int u = 0; u < AHEAD; ++u) {
          // (what does not move reads the pool's start: a load that may be left out would have all waits be for all loads)
          const int i = at + u * entries + entry;
          const Entry x = list[min(i, n - 1)];
          const bool go = i < n && e < per && x[0] >= 0;
          const int64_t from = ((int64_t)x[0] * c.heads + m.head) * stride + (int64_t)x[1] * row + e * (int)sizeof(T);
          data[round][u] = *reinterpret_cast<const T*>(base + (go ? from : 0));
          to[round][u] = go ? ((int64_t)x[2] * c.heads + m.head) * stride + (int64_t)x[3] * row + e * (int)sizeof(T) : -1;
        }
      };
      auto store = [&](int round) {
#pragma unroll
        for (int u = 0; u < AHEAD; ++u)
          if (to[round][u] >= 0) *reinterpret_cast<T*>(base + to[round][u]) = data[round][u];
      };
      load(0, 0);
      for (int at = 0; at < n; at += 2 * step) {
        load(1, at + step);
        __syncthreads();
        store(0);
        load(0, at + 2 * step);
        __syncthreads();
        store(1);
      }
    }
  }
  return bad;
}

// The scale bytes of a row, as wide as their place allows.
__device__ __forceinline__ void move_scales(const Cache& c, const Moves& m, Entry* list, uint8_t* base) {
  if (c.groups % 4 == 0)
    move_part<uint32_t, 4>(c, m, list, base, c.block, c.groups, c.groups / 4, 1);
  else if (c.groups % 2 == 0)
    move_part<uint16_t, 4>(c, m, list, base, c.block, c.groups, c.groups / 2, 1);
  else
    move_part<uint8_t, 4>(c, m, list, base, c.block, c.groups, c.groups, 1);
}

static __global__ __launch_bounds__(kKeepThreads) void k_keep(KeepArgs a) {
  const Cache& c = a.c;
  __shared__ Entry list[kKeepList];
  int id = blockIdx.x;
  const int part = id % a.parts;
  id /= a.parts;
  const int head = id % c.heads, b = id / c.heads;
  const int32_t told = c.lens[b];
  const int64_t cap = (int64_t)c.max_pages * c.page.by;
  Moves m;
  m.len = min(max(told, 0), (int)(cap < kMaxLen ? cap : kMaxLen));
  bool bad = m.len != told;
  m.first = 0;
  m.count = a.width;
  if (a.counts) {
    const int32_t n = a.counts[b];
    m.count = min(max(n, 0), a.width);
    bad |= n != m.count;
  }
  if (a.from_new) {
    // (what had to be cut leaves the first new token's place unknown: nothing moves)
    const int64_t n = (int64_t)c.starts[b + 1] - c.starts[b];
    const bool known = m.len == told && n >= 0 && n <= m.len;
    m.first = known ? m.len - (int)n : 0;
    m.count = known ? m.count : 0;
    bad |= !known;
  }
  m.keep = a.keep + ((int64_t)b * a.lists + (a.lists > 1 ? head : 0)) * a.width;
  m.table = c.table + (int64_t)b * c.max_pages;
  m.head = head;
  const int chunks = c.row / 16, codes = 2 * a.slices;
  if (part < codes) {
    const bool is_v = part >= a.slices;
    const int slice = is_v ? part - a.slices : part;
    uint8_t* base = c.pool + (is_v ? c.v_off : 0) + slice * a.side * 16;
    bad |= move_part<u32x4, kKeepAhead>(c, m, list, base, c.block, c.row, min(a.side, chunks - slice * a.side), a.side);
  } else if (part == codes && c.groups > 0) {
    move_scales(c, m, list, c.pool + c.ks_off);
    move_scales(c, m, list, c.pool + c.vs_off);
  } else {
    move_part<uint32_t, 4>(c, m, list, reinterpret_cast<uint8_t*>(a.weights), (int64_t)c.page.by * 4, 4, 1, 1);
  }
  if (a.err && part == 0 && __syncthreads_or(bad) && threadIdx.x == 0) atomicAdd(a.err, 1);
}

}  // namespace serve
