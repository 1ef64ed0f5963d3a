// The choice of the cached tokens that stay: of a sequence of m > budget tokens the first `sinks`, the last `recent`, and
// of those between the budget - sinks - recent of the largest weight, the lowest place of equals; each key head for itself.
//
// One workgroup a (sequence, key head), which holds the weights of up to 32768 (or 4096) places in registers as 32-bit numbers
// of the same order.  The smallest that stays is found digit by digit from the top (11, 11 and 10 bits: a histogram in LDS, its
// sums from the top, the bin that the wanted count falls into); everything above it stays, of its equals the first.  A wave
// holds consecutive places, four a lane and 256 in four rounds (a page number and, where pages allow it, one load serve four), so
// the places that stay are written in order after one scan over the waves' counts.
// Nothing is sorted, and the order of the histogram's atomics changes nothing.
//
// Measured: 4096 of up to 32768 places of 32 sequences and 8 heads 26 us, a compute unit each (12 of them the digits, 6 the
// places; the bytes alone are worth 5): what bounds it is the chain of barriers and scans behind one workgroup's loads, and their
// addresses; with a load a place it took 29.  2048 of 2304 for 8 heads 8 us.  Past 32768 places each digit reads all of them again:
// 4096 of 131000 for 8 heads 135 us.
#pragma once

#include "serve_common.h"

namespace serve {

struct ChooseArgs {
  Cache c;
  const float* weights;  // [pages][heads][page]
  int32_t* keep;         // [batch][heads][budget]
  int32_t* counts;       // [batch]
  int32_t budget, sinks, recent;
  bool fours;            // weights are aligned to 16 bytes and pages hold a multiple of four
  int32_t* err;
};

// A weight as a number of the same order.  NaN counts as the smallest, the zeros as one.
__device__ __forceinline__ uint32_t order_of(float w) {
  const float x = w != w ? -INFINITY : w + 0.0f;
  const uint32_t u = __float_as_uint(x);
  return u >> 31 ? ~u : u | 0x80000000u;
}

constexpr uint32_t kAlways = 0xffffffffu, kNever = 0;  // of places that stay in any case, and of none: no weight has these

constexpr int kChooseThreads = 1024, kChooseWaves = kChooseThreads / kWave;
constexpr int kDigit = 11, kBins = 1 << kDigit;

// Exclusive sums over the workgroup of one number a thread, in the threads' order.
__device__ __forceinline__ int scan_block(int x, int* waves) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int sum = x;
#pragma unroll
  for (int d = 1; d < kWave; d <<= 1) {
    const int y = __shfl_up(sum, d);
    if (lane >= d) sum += y;
  }
  if (lane == kWave - 1) waves[wave] = sum;
  __syncthreads();
  int before = 0;
#pragma unroll
  for (int i = 0; i < kChooseWaves; ++i) before += i < wave ? waves[i] : 0;
  return before + sum - x;
}

// HELD: places a thread holds.  LONG: sequences that pass that are read again for each digit, HELD rounds at a time.
template <int HELD, bool LONG>
__global__ __launch_bounds__(kChooseThreads) void k_choose(ChooseArgs a) {
  __shared__ int bins[kBins], waves[3][kChooseWaves], found[3][2];
  __shared__ int sure_of[2][kChooseWaves], same_of[2][kChooseWaves];  // (two: a wave may be a block of rounds ahead)
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
  bool lost = false;
  const int32_t* table = c.table + (int64_t)b * c.max_pages;
  if (len <= a.budget) {
    for (int i = tid; i < a.budget; i += kChooseThreads) keep[i] = i < len ? i : -1;
    if (a.err && head == 0) {  // no weight is read, but pages are counted as for the others
      const int pages = len > 0 ? (int)divide((uint32_t)(len - 1), c.page) + 1 : 0;
      for (int i = tid; i < pages; i += kChooseThreads) lost |= table[i] < 0 || table[i] >= c.pages;
      if (__any(lost) && lane == 0) atomicAdd(a.err, 1);
    }
    return;
  }
  const int low = a.sinks, high = len - a.recent;  // those between are chosen from
  int want = a.budget - a.sinks - a.recent;
  uint32_t held[HELD];
  const int rounds = (len + kChooseThreads - 1) / kChooseThreads;
  // A block of up to HELD rounds from r0 on: this thread's place in round i, and all their numbers.  All page numbers, then
  // all weights are under way at once (past the last place: that one's again).
  static_assert(HELD % 4 == 0, "four places a lane");
  auto rounds_of = [&](int r0) { return min((rounds - r0 + 3) & ~3, HELD); };  // of a block
  auto place_of = [&](int r0, int i) { return r0 * kChooseThreads + (wave * rounds_of(r0) + (i & ~3)) * kWave + lane * 4 + (i & 3); };
  auto hold = [&](int r0) {
    float w[HELD];
    bool gone[HELD / 4];
    if (a.fours) {
      int32_t ids[HELD / 4];
      int slots[HELD / 4];
#pragma unroll
      for (int q = 0; q < HELD / 4; ++q) {
        const uint32_t j = (uint32_t)min(place_of(r0, 4 * q), (len - 1) & ~3), page = divide(j, c.page);
        slots[q] = (int)(j - page * c.page.by);
        ids[q] = table[page];
      }
#pragma unroll
      for (int q = 0; q < HELD / 4; ++q) {
        gone[q] = ids[q] < 0 || ids[q] >= c.pages;
        lost |= gone[q];
        const f32x4 x = *reinterpret_cast<const f32x4*>(a.weights + ((int64_t)(gone[q] ? 0 : ids[q]) * c.heads + head) * c.page.by + slots[q]);
#pragma unroll
        for (int k = 0; k < 4; ++k) w[4 * q + k] = x[k];
      }
#pragma unroll
      for (int i = 0; i < HELD; ++i) w[i] = gone[i / 4] ? -INFINITY : w[i];
    } else {
      int32_t ids[HELD];
      int slots[HELD];
#pragma unroll
      for (int i = 0; i < HELD; ++i) {
        const uint32_t j = (uint32_t)min(place_of(r0, i), len - 1), page = divide(j, c.page);
        slots[i] = (int)(j - page * c.page.by);
        ids[i] = table[page];
      }
#pragma unroll
      for (int i = 0; i < HELD; ++i) {
        const bool ok = ids[i] >= 0 && ids[i] < c.pages;
        lost |= !ok;
        w[i] = a.weights[((int64_t)(ok ? ids[i] : 0) * c.heads + head) * c.page.by + slots[i]];
        if (!ok) slots[i] = -1;
      }
#pragma unroll
      for (int i = 0; i < HELD; ++i) w[i] = slots[i] < 0 ? -INFINITY : w[i];  // (no page counts as NaN does)
    }
#pragma unroll
    for (int i = 0; i < HELD; ++i) {
      const int j = place_of(r0, i);
      const uint32_t u = order_of(w[i]);
      held[i] = i >= rounds_of(r0) || j >= len ? kNever : j < low || j >= high ? kAlways : u;
    }
  };
  if (!LONG) hold(0);
  uint32_t least = kAlways - 1;  // the least that stays (nothing between does where nothing is wanted)
  if (want > 0) {
    uint32_t known = 0;  // digits found so far
    least = 0;
#pragma unroll LONG ? 1 : 3
    for (int digit = 0; digit < 3; ++digit) {
      const int shift = digit == 0 ? 21 : digit == 1 ? 10 : 0;
      const uint32_t mask = digit == 2 ? 1023u : 2047u;
      for (int i = tid; i < kBins; i += kChooseThreads) bins[i] = 0;
      __syncthreads();
      for (int r0 = 0; r0 < (LONG ? rounds : 1); r0 += HELD) {
        if (LONG) hold(r0);
#pragma unroll
        for (int i = 0; i < HELD; ++i)
          if (i < rounds_of(r0) && (held[i] & known) == least && (digit > 0 || (held[i] != kNever && held[i] != kAlways)))
            atomicAdd(&bins[held[i] >> shift & mask], 1);
      }
      __syncthreads();
      // two bins a thread, from the top
      const int top = kBins - 1 - 2 * tid, first = bins[top], second = bins[top - 1];
      const int above = scan_block(first + second, waves[digit]);
      if (above < want && want <= above + first) found[digit][0] = top, found[digit][1] = want - above;
      if (above + first < want && want <= above + first + second) found[digit][0] = top - 1, found[digit][1] = want - above - first;
      __syncthreads();
      least |= (uint32_t)found[digit][0] << shift;
      known |= mask << shift;
      want = found[digit][1];
    }
  }
  // the places in order, HELD rounds at a time; `want` of those equal to the least stay
  int sure_before = 0, same_before = 0;
  for (int r0 = 0, turn = 0; r0 < (LONG ? rounds : 1); r0 += HELD, turn ^= 1) {
    if (LONG) hold(r0);
    int sure = 0, same = 0;  // of this wave
#pragma unroll
    for (int i = 0; i < HELD; ++i) {
      if (i < rounds_of(r0)) {
        sure += __popcll(__ballot(held[i] > least));
        same += __popcll(__ballot(held[i] == least));
      }
    }
    if (lane == 0) sure_of[turn][wave] = sure, same_of[turn][wave] = same;
    __syncthreads();
    int sure_at = sure_before, same_at = same_before;
#pragma unroll
    for (int i = 0; i < kChooseWaves; ++i) {
      const int x = sure_of[turn][i], y = same_of[turn][i];
      sure_at += i < wave ? x : 0;
      same_at += i < wave ? y : 0;
      sure_before += x;
      same_before += y;
    }
    sure_at = __builtin_amdgcn_readfirstlane(sure_at);
    same_at = __builtin_amdgcn_readfirstlane(same_at);
    // (the masks are made again: kept, they would take more registers than there are)
#pragma unroll
    for (int i = 0; i < HELD; ++i) asm volatile("" : "+v"(held[i]));
#pragma unroll
    for (int q = 0; q < HELD / 4; ++q) {
      if (4 * q < rounds_of(r0)) {
        const uint64_t below = (1ull << lane) - 1;
        uint64_t above[4], equal[4];
        int mine = sure_at, equals = same_at;  // kept, and equal to the least, before this lane's first place
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          above[k] = __ballot(held[4 * q + k] > least);
          equal[k] = __ballot(held[4 * q + k] == least);
          mine += __popcll(above[k] & below);
          equals += __popcll(equal[k] & below);
          sure_at += __popcll(above[k]);
          same_at += __popcll(equal[k]);
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          // of the equals the first `want`: those before, all of them kept, move it on
          const bool is_above = held[4 * q + k] > least, is_equal = held[4 * q + k] == least;
          const int at = mine + min(equals, want);
          if ((is_above || (is_equal && equals < want)) && at < a.budget) keep[at] = place_of(r0, 4 * q + k);
          mine += is_above;
          equals += is_equal;
        }
      }
    }
  }
  if (a.err && __any(lost) && lane == 0) atomicAdd(a.err, 1);
}

}  // namespace serve
