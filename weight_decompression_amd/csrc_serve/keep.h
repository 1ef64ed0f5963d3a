// The move of the tokens that stay to the front of their sequence: place first + i takes what lies at first + keep[i],
// keep ascending, in place and for each key head by its own list.
//
// What moves is read once and written once; HBM bounds it for long lists, the launch for short ones.  A token's parts (key and
// value codes, their scale bytes, its weight) never meet, so a workgroup has one part of a (sequence, key head), of the
// codes 64 bytes of each row, and takes the list in order, a batch of entries at a time: all of a batch is read, then, after
// a barrier, written.  That is enough for moves in place: keep[i] >= i, so what a batch writes (its own i) lies before
// anything that later batches read (at or past their own, larger i), and what earlier batches read is past the barrier.  The
// loads of the next batch are under way while a batch is written.
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
  int32_t slices;         // of a row of codes
  int32_t parts;          // workgroups a (sequence, key head): slices of keys, slices of values, scales, weights
};

constexpr int kKeepThreads = 256, kKeepAhead = 4;

// The places of a list: of entry i where it comes from and where it goes, or nothing.
struct Moves {
  const int32_t* keep;
  const int32_t* table;
  int count, first, len;
};
__device__ __forceinline__ bool move_of(const Cache& c, const Moves& m, int i, int head, int64_t* from, int* from_slot, int64_t* to,
                                        int* to_slot, bool* bad) {
  if (i >= m.count) return false;
  const int k = m.keep[i];
  if (k == i || k == -1) return false;
  const bool fits = k > i && (i == 0 || k > m.keep[i - 1]) && k < m.len - m.first;
  if (!fits) {
    *bad = true;
    return false;
  }
  const uint32_t src = (uint32_t)(m.first + k), dst = (uint32_t)(m.first + i);
  const uint32_t sp = divide(src, c.page), dp = divide(dst, c.page);
  const int32_t s = m.table[sp], d = m.table[dp];
  if (s < 0 || s >= c.pages || d < 0 || d >= c.pages) {
    *bad = true;
    return false;
  }
  *from = (int64_t)s * c.heads + head;
  *to = (int64_t)d * c.heads + head;
  *from_slot = (int)(src - sp * c.page.by);
  *to_slot = (int)(dst - dp * c.page.by);
  return true;
}

// Moves `per` elements of T of every entry's row: element e of a token lies at base + block * stride + slot * row + e.
template <typename T>
__device__ __forceinline__ bool move_part(const Cache& c, const Moves& m, int head, uint8_t* base, int64_t stride, int row, int per) {
  const int tid = threadIdx.x;
  // elements of a row side by side: 1, 2 or 4 threads an entry, more elements one after the other
  const int side = per >= 4 ? 4 : per >= 2 ? 2 : 1;
  const int entry = tid / side, lane = tid % side, entries = kKeepThreads / side;
  bool bad = false;
  for (int e0 = 0; e0 < per; e0 += side) {
    const int e = e0 + lane;
    T data[2][kKeepAhead];
    int64_t to[2][kKeepAhead];
    auto load = [&](int round, int i0) {
#pragma unroll
      for (int u = 0; u < kKeepAhead; ++u) {
        int64_t sb, db;
        int ss, ds;
        to[round][u] = -1;
        if (move_of(c, m, i0 + u * entries + entry, head, &sb, &ss, &db, &ds, &bad) && e < per) {
          data[round][u] = *reinterpret_cast<const T*>(base + sb * stride + (int64_t)ss * row + e * (int)sizeof(T));
          to[round][u] = db * stride + (int64_t)ds * row + e * (int)sizeof(T);
        }
      }
    };
    auto store = [&](int round) {
#pragma unroll
      for (int u = 0; u < kKeepAhead; ++u)
        if (to[round][u] >= 0) *reinterpret_cast<T*>(base + to[round][u]) = data[round][u];
    };
    const int step = entries * kKeepAhead;
    load(0, 0);
    for (int i0 = 0; i0 < m.count; i0 += 2 * step) {
      load(1, i0 + step);
      __syncthreads();
      store(0);
      load(0, i0 + 2 * step);
      __syncthreads();
      store(1);
    }
  }
  return bad;
}

static __global__ __launch_bounds__(kKeepThreads) void k_keep(KeepArgs a) {
  const Cache& c = a.c;
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
  if (a.from_new) {
    const int64_t n = (int64_t)c.starts[b + 1] - c.starts[b];
    const int cut = (int)(n < 0 ? 0 : n > m.len ? m.len : n);
    bad |= n != cut;
    m.first = m.len - cut;
  }
  m.count = a.width;
  if (a.counts) {
    const int32_t n = a.counts[b];
    m.count = min(max(n, 0), a.width);
    bad |= n != m.count;
  }
  m.keep = a.keep + ((int64_t)b * a.lists + (a.lists > 1 ? head : 0)) * a.width;
  m.table = c.table + (int64_t)b * c.max_pages;
  const int chunks = c.row / 16, codes = 2 * a.slices;
  if (part < codes) {
    const bool is_v = part >= a.slices;
    const int slice = is_v ? part - a.slices : part;
    uint8_t* base = c.pool + (is_v ? c.v_off : 0) + slice * 64;
    bad |= move_part<u32x4>(c, m, head, base, c.block, c.row, min(4, chunks - slice * 4));
  } else if (part == codes && c.groups > 0) {
    uint8_t* ks = c.pool + c.ks_off;
    uint8_t* vs = c.pool + c.vs_off;
    if (c.groups % 4 == 0) {
      move_part<uint32_t>(c, m, head, ks, c.block, c.groups, c.groups / 4);
      move_part<uint32_t>(c, m, head, vs, c.block, c.groups, c.groups / 4);
    } else if (c.groups % 2 == 0) {
      move_part<uint16_t>(c, m, head, ks, c.block, c.groups, c.groups / 2);
      move_part<uint16_t>(c, m, head, vs, c.block, c.groups, c.groups / 2);
    } else {
      move_part<uint8_t>(c, m, head, ks, c.block, c.groups, c.groups);
      move_part<uint8_t>(c, m, head, vs, c.block, c.groups, c.groups);
    }
  } else {
    uint8_t* w = reinterpret_cast<uint8_t*>(a.weights);
    move_part<uint32_t>(c, m, head, w, (int64_t)c.page.by * 4, 4, 1);
  }
  if (a.err && part == 0 && __syncthreads_or(bad) && threadIdx.x == 0) atomicAdd(a.err, 1);
}

}  // namespace serve
