// The check of drafted trees.  At a node whose children were picked (not drawn) in some order, the target's token is
// one of theirs with the target's own probabilities: child i is taken while u_i S < p(x_i), where S = 1 - the p of the
// children refused before it, so that its chance is p(x_i) / S among what is left; a refused token cannot come again.  Where
// no child is taken, one token is drawn from p without the refused, as the check of drafts draws (argmax of p_v / e_v).
// S and its products are in 64 bits: a probability's 24 bits and the sums of up to 63 of them lose nothing that a
// comparison with a 24-bit p could show but in the last few of 2^53 cases.
//
// A sequence's nodes fit a wave: lane i holds node i, its parent, token, u and the parent's probability of its token,
// one gather for all of them.  The walk then touches no memory: a node's children are a ballot, each step reads one lane.
// Every workgroup of a sequence walks by itself, then takes its share of the row that the token is drawn from: that
// row and its noise, read once, are what the check cannot do without (HBM bounds it for many sequences, two launches and a
// chain of four loads, starts -> parents and tokens -> probabilities -> row, for few).  Measured: 96 trees of up to 32 nodes
// over 100003 entries in f32 19.5 us, 3.9 TB/s, where a large copy reaches 5.1 (17 us are left when the row is not read); one of
// 16 over 32000: 7 us and the second launch 2.
#pragma once

#include "draft.h"

namespace serve {

struct TreeArgs {
  const void* target;       // [nodes][vocab]
  const int32_t* starts;    // [batch + 1]
  const int32_t* tokens;    // [nodes]
  const int32_t* parents;   // [nodes]
  const float* uniforms;    // [nodes]
  const float* noise;       // [batch][vocab]
  uint64_t* keys;           // [batch][parts]
  int32_t* accepted;        // [batch]
  int32_t* path;            // [batch][width]
  int32_t* out;             // [batch][width]
  int32_t* err;
  int32_t batch, nodes, vocab, width, parts, per;
};

// What the walk of a sequence finds, the same in every lane but for token.
struct Walk {
  uint64_t path, refused;  // nodes on the way, and the last one's children that were not taken
  int64_t row;             // of the last node
  int token;               // of this lane's node
  bool any, bad;           // whether there is a node; what is counted
};

__device__ __forceinline__ double lane_f64(double x, int lane) {
  const uint64_t u = __builtin_bit_cast(uint64_t, x);
  return __builtin_bit_cast(double, (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)u, lane) |
                                        (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(u >> 32), lane) << 32);
}

template <bool F32>
__device__ __forceinline__ Walk walk_of(const TreeArgs& a, int b) {
  const int lane = threadIdx.x & 63;
  const int32_t s0 = a.starts[b], s1 = a.starts[b + 1];
  const int first = min(max(s0, 0), a.nodes), all = min(max(s1, first), a.nodes) - first;
  const int n = min(all, LLVQ_MAX_NODES);
  Walk w;
  w.any = n > 0;
  w.bad = s0 != first || s1 != first + n;
  const bool in = lane < n;
  w.token = in ? a.tokens[first + lane] : -1;
  int up = in ? a.parents[first + lane] : -1;
  const bool stray = up < -1 || up >= lane, outside = in && lane > 0 && (w.token < 0 || w.token >= a.vocab);
  w.bad |= __any((in && stray) || outside) != 0;
  if (stray) up = -1;
  double p = 0.0, u = 0.0;
  if (in && up >= 0 && !outside) {
    const float x = prob<F32>(a.target, (int64_t)(first + up) * a.vocab + w.token);
    p = x > 0.0f ? (double)x : 0.0;  // (what is never drawn is never taken: NaN, negative)
    u = (double)a.uniforms[first + lane];
  }
  int cur = 0, length = 1;
  double left = 1.0;
  w.path = w.any ? 1 : 0;
  w.refused = 0;
  uint64_t todo = __ballot(up == 0);
  while (todo && length < a.width) {
    const int i = __builtin_ctzll(todo);
    todo &= todo - 1;
    const int x = __builtin_amdgcn_readlane(w.token, i);
    const bool again = (__ballot(w.token == x) & w.refused) != 0;
    const double pi = again ? 0.0 : lane_f64(p, i);
    if (lane_f64(u, i) * (left > 0.0 ? left : 0.0) < pi) {
      cur = i;
      ++length;
      left = 1.0;
      w.path |= 1ull << i;
      w.refused = 0;
      todo = __ballot(up == i);
    } else {
      left -= pi;
      w.refused |= 1ull << i;
    }
  }
  w.row = (int64_t)(first + cur) * a.vocab;
  return w;
}

// A workgroup's best of entries [from, end) of the row, in every thread.  The refused tokens are looked for only where an
// entry may be the best so far and shares its last six bits with one of them: the first entries of every thread may all be
// (96 trees of up to 32 nodes over 100003 entries: 20.4 us without the bits, 19.5 with them).  After its first entries a lane
// only looks at what may pass the best of its wave (24.7 us by its own best): entries come in ascending order, so an equal one
// has lost.
template <bool F32, int THREADS>
__device__ __forceinline__ uint64_t best_left(const TreeArgs& a, int b, const Walk& w, bool without, int64_t from, int64_t end) {
  constexpr int kAhead = THREADS == 1024 ? 16 : 8;
  __shared__ uint64_t best[THREADS / 64];
  __shared__ int gone[kWave];
  const int tid = threadIdx.x;
  const int many = without ? __popcll(w.refused) : 0;
  __syncthreads();  // (an earlier call's shared values have been read)
  if (tid < kWave && (w.refused >> tid & 1)) gone[__popcll(w.refused & ((1ull << tid) - 1))] = w.token;
  __syncthreads();
  uint64_t bits = without && (w.refused >> (tid & 63) & 1) ? 1ull << (w.token & 63) : 0;
#pragma unroll
  for (int d = 1; d < kWave; d <<= 1) bits |= (uint64_t)__shfl_xor((unsigned long long)bits, d);
  auto refused = [&](int v) {
    if (!(bits >> (v & 63) & 1)) return false;
    for (int i = 0; i < many; ++i)
      if (gone[i] == v) return true;
    return false;
  };
  const float* noise = a.noise + (int64_t)b * a.vocab;
  Best mine, wave_best;
  for (int64_t v0 = from + tid; v0 < end; v0 += THREADS * kAhead) {
    float p[kAhead], e[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int64_t v = min(v0 + THREADS * i, end - 1);  // (loads that may be left out would be waited for one by one)
      p[i] = prob<F32>(a.target, w.row + v);
      e[i] = noise[v];
    }
    bool any = false;
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      p[i] = v0 + THREADS * i < end ? p[i] : 0.0f;
      any |= wave_best.may(p[i], e[i]);
    }
    if (any) {
#pragma unroll
      for (int i = 0; i < kAhead; ++i)
        if (wave_best.may(p[i], e[i]) && !refused((int)(v0 + THREADS * i))) mine.take(p[i], e[i], (int)(v0 + THREADS * i));
    }
    if (__any(mine.score > wave_best.score)) {
      wave_best.score = mine.score;
#pragma unroll
      for (int d = 1; d < kWave; d <<= 1) wave_best.score = fmaxf(wave_best.score, __shfl_xor(wave_best.score, d));
    }
  }
  const uint64_t k = wave_max(mine.key());
  if ((tid & 63) == 0) best[tid >> 6] = k;
  __syncthreads();
  uint64_t top = best[0];
  for (int i = 1; i < THREADS / 64; ++i) top = best[i] > top ? best[i] : top;
  return top;
}

// The path and tokens of sequence b, all but the drawn one.
__device__ __forceinline__ void write_path(const TreeArgs& a, int b, const Walk& w, int threads) {
  const int tid = threadIdx.x, length = __popcll(w.path);
  const int64_t at = (int64_t)b * a.width;
  for (int i = tid; i < a.width; i += threads)
    if (i >= length) {
      a.path[at + i] = -1;
      a.out[at + i] = -1;
    }
  if (tid < kWave && (w.path >> tid & 1)) {
    const int i = __popcll(w.path & ((1ull << tid) - 1));
    a.path[at + i] = tid;
    if (i > 0) a.out[at + i - 1] = w.token;
  }
  if (tid == 0) {
    a.accepted[b] = w.any ? length - 1 : 0;
    if (a.err && w.bad) atomicAdd(a.err, 1);
  }
}
// The drawn token of a sequence that accepted that many drafts.
__device__ __forceinline__ void write_drawn(const TreeArgs& a, int b, int accepted, uint64_t k) {
  if (threadIdx.x != 0) return;
  a.out[(int64_t)b * a.width + accepted] = k ? (int)(0xffffffffu - (uint32_t)k) : -1;
  if (a.err && !k) atomicAdd(a.err, 1);
}

// Where nothing but the refused is left, the draw is from all of p.
template <bool F32>
__global__ __launch_bounds__(1024) void k_tree_one(TreeArgs a) {
  const int b = blockIdx.x;
  const Walk w = walk_of<F32>(a, b);
  write_path(a, b, w, 1024);
  if (!w.any) return;
  uint64_t k = best_left<F32, 1024>(a, b, w, true, 0, a.vocab);
  if (k == 0) k = best_left<F32, 1024>(a, b, w, false, 0, a.vocab);
  write_drawn(a, b, __popcll(w.path) - 1, k);
}

template <bool F32>
__global__ __launch_bounds__(256) void k_tree_part(TreeArgs a) {
  const int b = blockIdx.y;
  const Walk w = walk_of<F32>(a, b);
  if (blockIdx.x == 0) write_path(a, b, w, 256);
  if (!w.any) return;
  const int64_t from = (int64_t)blockIdx.x * a.per;
  const uint64_t k = best_left<F32, 256>(a, b, w, true, from, min(from + a.per, (int64_t)a.vocab));
  if (threadIdx.x == 0) a.keys[(int64_t)b * a.parts + blockIdx.x] = k;
}

// The best of the parts; the walk is only taken again where there is none.
template <bool F32>
__global__ __launch_bounds__(256) void k_tree_pick(TreeArgs a) {
  const int b = blockIdx.x;
  if (a.path[(int64_t)b * a.width] < 0) return;  // no nodes
  const int accepted = a.accepted[b];
  uint64_t k = 0;
  for (int i = threadIdx.x & 63; i < a.parts; i += 64) {
    const uint64_t x = a.keys[(int64_t)b * a.parts + i];
    k = x > k ? x : k;
  }
  k = wave_max(k);  // (the same in every wave)
  if (k == 0) k = best_left<F32, 256>(a, b, walk_of<F32>(a, b), false, 0, a.vocab);
  write_drawn(a, b, accepted, k);
}

}  // namespace serve
