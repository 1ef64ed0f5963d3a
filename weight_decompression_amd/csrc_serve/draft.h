// The check of drafted tokens.  Draft i of a sequence, drawn from q_i, is accepted while
// u_i q_i(x_i) < p_i(x_i) (u uniform in [0, 1): with probability min(1, p / q)); the first one that is not
// is replaced by a token drawn from the rest, max(p - q, 0), and after all of them one more is drawn from p.
// A draw from weights w is argmax_v w_v / e_v with e exponential: the race whose winner is v with
// probability w_v / sum w.  It needs no sum, so no order of summation can change a token.
//
// Only the row that the sequence draws from is read: p, q and e once, which HBM bounds for many sequences
// and the launches for few.  The vocabulary is split over workgroups; each finds the first
// unaccepted draft by itself (a few scalars) and leaves one key for each of the two draws (the rest, and p alone for
// the case that the rest is empty): the score's bits above the complement of the index, so that
// the largest key is the best score at the lowest index.  The second kernel takes the largest.
#pragma once

#include "serve_common.h"

namespace serve {

constexpr int kMaxDrafts = 64;

struct DraftArgs {
  const void* target;       // [batch][drafts + 1][vocab]
  const void* draft;        // [batch][drafts][vocab], or null: every draft was certain
  const int32_t* tokens;    // [batch][drafts]
  const int32_t* counts;    // [batch] or null
  const float* uniforms;    // [batch][drafts]
  const float* noise;       // [batch][vocab]
  uint64_t* keys;           // [batch][parts][2]
  int32_t* accepted;
  int32_t* out;             // [batch][drafts + 1]
  int32_t* err;
  int32_t batch, drafts, vocab, parts, per;  // per: entries of a part
};

template <bool F32>
__device__ __forceinline__ float prob(const void* p, int64_t at) {
  if constexpr (F32)
    return static_cast<const float*>(p)[at];
  else
    return bf16_f32(static_cast<const uint16_t*>(p)[at]);
}

// Accepted drafts of sequence b; the same in every lane of a wave.
template <bool F32>
__device__ __forceinline__ int accepted_of(const DraftArgs& a, int b, bool* bad) {
  const int lane = threadIdx.x & 63;
  const int n = a.counts ? min(max(a.counts[b], 0), a.drafts) : a.drafts;
  bool ok = false, wrong = a.counts && n != a.counts[b];
  if (lane < n) {
    const int64_t i = (int64_t)b * a.drafts + lane;
    const int x = a.tokens[i];
    if (x >= 0 && x < a.vocab) {
      const float p = prob<F32>(a.target, ((int64_t)b * (a.drafts + 1) + lane) * a.vocab + x);
      const float q = a.draft ? prob<F32>(a.draft, i * a.vocab + x) : 1.0f;
      ok = a.uniforms[i] * q < p;
    } else {
      wrong = true;
    }
  }
  *bad = __any(wrong);
  const uint64_t no = ~__ballot(ok);
  return no ? __builtin_ctzll(no) : kWave;
}

__device__ __forceinline__ uint64_t score_key(float w, float e, int v) {
  if (!(w > 0.0f) || !(e >= 0.0f)) return 0;
  const float s = __fdiv_rn(w, e);
  if (!(s >= 0.0f)) return 0;
  // bit 31 (a score has no sign) marks the key as one of a candidate
  return (uint64_t)(__float_as_uint(s) | 0x80000000u) << 32 | (0xffffffffu - (uint32_t)v);
}

__device__ __forceinline__ uint64_t wave_max(uint64_t k) {
#pragma unroll
  for (int d = 32; d; d >>= 1) {
    const uint64_t o = (uint64_t)__shfl_xor((unsigned long long)k, d);
    k = o > k ? o : k;
  }
  return k;
}

template <bool F32>
__global__ __launch_bounds__(256) void k_draft_part(DraftArgs a) {
  const int b = blockIdx.y, part = blockIdx.x, tid = threadIdx.x;
  bool bad;
  const int done = accepted_of<F32>(a, b, &bad);
  const int n = a.counts ? min(max(a.counts[b], 0), a.drafts) : a.drafts;
  const bool all = done >= n;
  const int64_t row = ((int64_t)b * (a.drafts + 1) + done) * a.vocab;
  const int64_t qrow = ((int64_t)b * a.drafts + done) * a.vocab;
  const int certain = !all && !a.draft ? a.tokens[(int64_t)b * a.drafts + done] : -1;
  const bool take = !all && a.draft;
  const int64_t from = (int64_t)part * a.per;
  const int64_t end = min(from + a.per, (int64_t)a.vocab);
  uint64_t rest = 0, plain = 0;
  for (int64_t v = from + tid; v < end; v += 256) {
    const float p = prob<F32>(a.target, row + v);
    const float e = a.noise[(int64_t)b * a.vocab + v];
    float w = p;
    if (take) w -= prob<F32>(a.draft, qrow + v);
    if ((int)v == certain) w = 0.0f;
    const uint64_t kr = score_key(w, e, (int)v), kp = score_key(p, e, (int)v);
    rest = kr > rest ? kr : rest;
    plain = kp > plain ? kp : plain;
  }
  __shared__ uint64_t best[2][4];
  rest = wave_max(rest);
  plain = wave_max(plain);
  if ((tid & 63) == 0) best[0][tid >> 6] = rest, best[1][tid >> 6] = plain;
  __syncthreads();
  if (tid < 2) {
    uint64_t k = 0;
    for (int i = 0; i < 4; ++i) k = best[tid][i] > k ? best[tid][i] : k;
    a.keys[((int64_t)b * a.parts + part) * 2 + tid] = k;
  }
}

template <bool F32>
__global__ __launch_bounds__(64) void k_draft_pick(DraftArgs a) {
  const int b = blockIdx.x, lane = threadIdx.x;
  bool bad;
  const int done = accepted_of<F32>(a, b, &bad);
  uint64_t rest = 0, plain = 0;
  for (int i = lane; i < a.parts; i += 64) {
    const uint64_t* k = a.keys + ((int64_t)b * a.parts + i) * 2;
    rest = k[0] > rest ? k[0] : rest;
    plain = k[1] > plain ? k[1] : plain;
  }
  rest = wave_max(rest);
  plain = wave_max(plain);
  const uint64_t k = rest ? rest : plain;
  const int last = k ? (int)(0xffffffffu - (uint32_t)k) : -1;
  for (int i = lane; i <= a.drafts; i += 64)
    a.out[(int64_t)b * (a.drafts + 1) + i] = i < done ? a.tokens[(int64_t)b * a.drafts + i] : i == done ? last : -1;
  if (lane == 0) {
    a.accepted[b] = done;
    if (a.err && (bad || !k)) atomicAdd(a.err, 1);
  }
}

}  // namespace serve
