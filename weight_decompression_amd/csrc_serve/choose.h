// The choice of the cached tokens that stay: of a sequence of m > budget tokens the first `sinks`, the last `recent`, and
// of those between the budget - sinks - recent of the largest weight, the lowest place of equals; each key head for itself.
//
// One workgroup a (sequence, key head).  The weights become 32-bit numbers of the same order; the smallest that stays is
// found digit by digit from the top (11, 11 and 10 bits: a histogram in LDS, its sums from the top, the bin that the wanted
// count falls into), and everything above it stays, of its equals the first.  The places are then written in order: every
// wave counts its 64 places of each round of 1024, one scan over the rounds and waves gives each wave where it writes.
// Nothing is sorted, and the order of the histogram's atomics changes nothing.
#pragma once

#include "serve_common.h"

namespace serve {

struct ChooseArgs {
  Cache c;
  const float* weights;  // [pages][heads][page]
  int32_t* keep;         // [batch][heads][budget]
  int32_t* counts;       // [batch]
  int32_t budget, sinks, recent;
  int32_t* err;
};

// A weight as a number of the same order.  NaN counts as the smallest, the zeros as one.
__device__ __forceinline__ uint32_t order_of(float w) {
  const float x = w != w ? -INFINITY : w + 0.0f;
  const uint32_t u = __float_as_uint(x);
  return u >> 31 ? ~u : u | 0x80000000u;
}

constexpr int kChooseThreads = 1024, kChooseWaves = kChooseThreads / kWave;
constexpr int kDigit = 11, kBins = 1 << kDigit;

// Exclusive sums over the workgroup of one number a thread, in the threads' order; *all: the sum of all.
__device__ __forceinline__ int scan_block(int x, int* waves, int* all) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int sum = x;
#pragma unroll
  for (int d = 1; d < kWave; d <<= 1) {
    const int y = __shfl_up(sum, d);
    if (lane >= d) sum += y;
  }
  __syncthreads();
  if (lane == kWave - 1) waves[wave] = sum;
  __syncthreads();
  int before = 0, total = 0;
#pragma unroll
  for (int i = 0; i < kChooseWaves; ++i) {
    const int w = waves[i];
    before += i < wave ? w : 0;
    total += w;
  }
  *all = total;
  return before + sum - x;
}

// HELD: places a thread holds; longer sequences are read again in each round.
template <int HELD>
__global__ __launch_bounds__(kChooseThreads) void k_choose(ChooseArgs a) {
  __shared__ int bins[kBins], waves[kChooseWaves], found[2];
  const Cache& c = a.c;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int head = (int)blockIdx.x % c.heads, b = (int)blockIdx.x / c.heads;
  const int32_t told = c.lens[b];
  const int64_t cap = (int64_t)c.max_pages * c.page.by;
  const int len = min(max(told, 0), (int)(cap < kMaxLen ? cap : kMaxLen));
  const int kept = min(len, a.budget);
  int32_t* keep = a.keep + ((int64_t)b * c.heads + head) * a.budget;
  if (head == 0 && tid == 0) {
    a.counts[b] = kept;
    if (a.err && len != told) atomicAdd(a.err, 1);
  }
  if (len <= a.budget) {
    for (int i = tid; i < a.budget; i += kChooseThreads) keep[i] = i < len ? i : -1;
    return;
  }
  bool lost = false;
  const int32_t* table = c.table + (int64_t)b * c.max_pages;
  auto weight_at = [&](int j) -> uint32_t {
    const uint32_t page = divide((uint32_t)j, c.page);
    const int32_t id = table[page];
    if (id < 0 || id >= c.pages) {  // (counts as NaN does)
      lost = true;
      return order_of(-INFINITY);
    }
    return order_of(a.weights[((int64_t)id * c.heads + head) * c.page.by + (j - page * c.page.by)]);
  };
  const int low = a.sinks, high = len - a.recent;  // those between are chosen from
  int want = a.budget - a.sinks - a.recent;
  uint32_t held[HELD];
  const int rounds = (len + kChooseThreads - 1) / kChooseThreads;
  const bool all_held = rounds <= HELD;
  if (all_held) {
#pragma unroll
    for (int i = 0; i < HELD; ++i) {
      const int j = i * kChooseThreads + tid;
      held[i] = j >= low && j < high ? weight_at(j) : 0;
    }
  }
  // runs f(place, weight's number) over this thread's places between
  auto each = [&](auto f) {
    if (all_held) {
#pragma unroll
      for (int i = 0; i < HELD; ++i) {
        const int j = i * kChooseThreads + tid;
        if (j >= low && j < high) f(j, held[i]);
      }
    } else {
      for (int i = 0; i < rounds; ++i) {
        const int j = i * kChooseThreads + tid;
        if (j >= low && j < high) f(j, weight_at(j));
      }
    }
  };
  uint32_t least = 0, known = 0;  // digits found so far
  int equal = 0;                  // of those with `least`, how many stay
  if (want > 0) {
#pragma unroll
    for (int digit = 0; digit < 3; ++digit) {
      const int shift = digit == 0 ? 21 : digit == 1 ? 10 : 0;
      const uint32_t mask = digit == 2 ? 1023u : 2047u;
      for (int i = tid; i < kBins; i += kChooseThreads) bins[i] = 0;
      __syncthreads();
      each([&](int, uint32_t u) {
        if ((u & known) == least) atomicAdd(&bins[u >> shift & mask], 1);
      });
      __syncthreads();
      // two bins a thread, from the top
      const int top = kBins - 1 - 2 * tid, first = bins[top], second = bins[top - 1];
      int all;
      const int above = scan_block(first + second, waves, &all);
      if (above < want && want <= above + first) found[0] = top, found[1] = want - above;
      if (above + first < want && want <= above + first + second) found[0] = top - 1, found[1] = want - above - first;
      __syncthreads();
      least |= (uint32_t)found[0] << shift;
      known |= mask << shift;
      want = found[1];
    }
    equal = want;
  } else {
    least = 0xffffffffu;  // nothing between stays
    known = 0xffffffffu;
  }
  // the places, in order, a round of 1024 at a time
  int done = 0, same = 0;  // kept, and equal to the least, in the rounds before
  auto write = [&](int i, uint32_t u) {
    const int j = i * kChooseThreads + tid;
    const bool between = j >= low && j < high;
    const bool is_same = between && u == least && equal > 0;
    const bool sure = j < len && (!between || u > least);
    int all, all_same;
    const int before_same = same + scan_block(is_same ? 1 : 0, waves, &all_same);
    const bool stays = sure || (is_same && before_same < equal);
    const int at = done + scan_block(stays ? 1 : 0, waves, &all);
    if (stays && at < a.budget) keep[at] = j;
    done += all;
    same += all_same;
  };
  if (all_held) {
#pragma unroll
    for (int i = 0; i < HELD; ++i)
      if (i < rounds) write(i, held[i]);
  } else {
    for (int i = 0; i < rounds; ++i) {
      const int j = i * kChooseThreads + tid;
      write(i, j >= low && j < high ? weight_at(j) : 0);
    }
  }
  if (a.err && __any(lost) && lane == 0 && wave >= 0) atomicAdd(a.err, 1);
}

}  // namespace serve
