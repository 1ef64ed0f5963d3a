// The choice of the cached tokens that stay: of a sequence of m > budget tokens the first `sinks`, the last `recent`, and
// of those between the budget - sinks - recent of the largest weight, the lowest place of equals; each key head for itself.
//
// One workgroup a (sequence, key head), which holds the weights of up to 32768 (or 4096) places in registers as 32-bit numbers
// of the same order.  The smallest that stays is found digit by digit from the top (11, 11 and 10 bits: a histogram in LDS, its
// sums from the top, the bin that the wanted count falls into); everything above it stays, of its equals the first.  The
// places are then written in order: each wave counts its 64 places of every round of 1024, one scan over all of these counts
// tells each wave where it writes.  Nothing is sorted, and the order of the histogram's atomics changes nothing.
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

// Exclusive sums over the workgroup of one number a thread, in the threads' order; *all: the sum of all.  A T may hold two
// counts side by side.
template <typename T>
__device__ __forceinline__ T scan_block(T x, T* waves, T* all) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  T sum = x;
#pragma unroll
  for (int d = 1; d < kWave; d <<= 1) {
    const T y = __shfl_up(sum, d);
    if (lane >= d) sum += y;
  }
  if (lane == kWave - 1) waves[wave] = sum;
  __syncthreads();
  T before = 0, total = 0;
#pragma unroll
  for (int i = 0; i < kChooseWaves; ++i) {
    const T w = waves[i];
    before += i < wave ? w : 0;
    total += w;
  }
  *all = total;
  return before + sum - x;
}

// HELD: places a thread holds.  LONG: sequences that pass that are read again for each digit, HELD rounds at a time.
template <int HELD, bool LONG>
__global__ __launch_bounds__(kChooseThreads) void k_choose(ChooseArgs a) {
  using Pair = unsigned long long;  // places that stay for sure, and from bit 32 on those equal to the least
  __shared__ int bins[kBins], waves[3][kChooseWaves], found[3][2];
  __shared__ Pair counts[HELD * kChooseWaves], pair_waves[kChooseWaves];
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
  const int low = a.sinks, high = len - a.recent;  // those between are chosen from
  int want = a.budget - a.sinks - a.recent;
  uint32_t held[HELD];
  const int rounds = (len + kChooseThreads - 1) / kChooseThreads;
  // all page numbers, then all weights under way at once (past the last place: that one's again)
  auto hold = [&](int r0) {
    int32_t ids[HELD];
    int slots[HELD];
#pragma unroll
    for (int i = 0; i < HELD; ++i) {
      const uint32_t j = (uint32_t)min((r0 + i) * kChooseThreads + tid, len - 1), page = divide(j, c.page);
      slots[i] = (int)(j - page * c.page.by);
      ids[i] = table[page];
    }
    float w[HELD];
#pragma unroll
    for (int i = 0; i < HELD; ++i) {
      const bool ok = ids[i] >= 0 && ids[i] < c.pages;
      lost |= !ok;
      w[i] = a.weights[((int64_t)(ok ? ids[i] : 0) * c.heads + head) * c.page.by + slots[i]];
      if (!ok) slots[i] = -1;
    }
#pragma unroll
    for (int i = 0; i < HELD; ++i) held[i] = order_of(slots[i] < 0 ? -INFINITY : w[i]);  // (no place counts as NaN does)
  };
  if (!LONG) hold(0);
  uint32_t least = 0xffffffffu;  // the least that stays (nothing between does where nothing is wanted)
  if (want > 0) {
    uint32_t known = 0;  // digits found so far
    least = 0;
#pragma unroll LONG ? 1 : 3
    for (int digit = 0; digit < 3; ++digit) {
      const int shift = digit == 0 ? 21 : digit == 1 ? 10 : 0;
      const uint32_t mask = digit == 2 ? 1023u : 2047u;
      for (int i = tid; i < kBins; i += kChooseThreads) bins[i] = 0;
      __syncthreads();
      auto count = [&](int j, uint32_t u) {
        if (j >= low && j < high && (u & known) == least) atomicAdd(&bins[u >> shift & mask], 1);
      };
      for (int r0 = 0; r0 < (LONG ? rounds : 1); r0 += HELD) {
        if (LONG) hold(r0);
#pragma unroll
        for (int i = 0; i < HELD; ++i)
          if (r0 + i < rounds) count((r0 + i) * kChooseThreads + tid, held[i]);
      }
      __syncthreads();
      // two bins a thread, from the top
      const int top = kBins - 1 - 2 * tid, first = bins[top], second = bins[top - 1];
      int all;
      const int above = scan_block(first + second, waves[digit], &all);
      if (above < want && want <= above + first) found[digit][0] = top, found[digit][1] = want - above;
      if (above + first < want && want <= above + first + second) found[digit][0] = top - 1, found[digit][1] = want - above - first;
      __syncthreads();
      least |= (uint32_t)found[digit][0] << shift;
      known |= mask << shift;
      want = found[digit][1];
    }
  }
  // the places in order, HELD rounds at a time; `want` of those equal to the least stay
  Pair before = 0;
  auto of = [&](int j, uint32_t u, uint64_t* sure, uint64_t* same) {
    const bool between = j >= low && j < high;
    *sure = __ballot(j < len && (!between || u > least));
    *same = __ballot(between && u == least && want > 0);
  };
  for (int r0 = 0; r0 < (LONG ? rounds : 1); r0 += HELD) {
    if (LONG) hold(r0);
#pragma unroll
    for (int i = 0; i < HELD; ++i) {
      if (r0 + i < rounds) {
        uint64_t sure, same;
        of((r0 + i) * kChooseThreads + tid, held[i], &sure, &same);
        if (lane == 0) counts[i * kChooseWaves + wave] = (Pair)__popcll(sure) | (Pair)__popcll(same) << 32;
      } else if (lane == 0) {
        counts[i * kChooseWaves + wave] = 0;
      }
    }
    __syncthreads();
    constexpr int kEach = (HELD * kChooseWaves + kChooseThreads - 1) / kChooseThreads;
    static_assert(kEach == 1, "a thread has one count");
    // (the masks are made again: kept, they would take more registers than there are)
#pragma unroll
    for (int i = 0; i < HELD; ++i) asm volatile("" : "+v"(held[i]));
    Pair all;
    const Pair mine = tid < HELD * kChooseWaves ? counts[tid] : 0, at = before + scan_block(mine, pair_waves, &all);
    if (tid < HELD * kChooseWaves) counts[tid] = at;
    before += all;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < HELD; ++i) {
      if (r0 + i < rounds) {
        const int j = (r0 + i) * kChooseThreads + tid;
        uint64_t sure, same;
        of(j, held[i], &sure, &same);
        const Pair from = counts[i * kChooseWaves + wave];
        const int same_before = (int)(from >> 32);
        const uint64_t below = (1ull << lane) - 1;
        // of the equals of this wave and round, the first few
        const bool taken = (same >> lane & 1) && same_before + __popcll(same & below) < want;
        const bool stays = (sure >> lane & 1) || taken;
        const int place = (int)(uint32_t)from + min(same_before, want) + __popcll(__ballot(stays) & below);
        if (stays && place < a.budget) keep[place] = j;
      }
    }
    __syncthreads();
  }
  if (a.err && __any(lost) && lane == 0) atomicAdd(a.err, 1);
}

}  // namespace serve
