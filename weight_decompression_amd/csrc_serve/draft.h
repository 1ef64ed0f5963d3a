// The check of drafted tokens.  Draft i of a sequence, drawn from q_i, is accepted while u_i q_i(x_i) <
// p_i(x_i) (u uniform in [0, 1): with probability min(1, p / q)); the first one that is not is replaced by
// a token drawn from the rest, max(p - q, 0), and after all of them one more is drawn from p. A draw from
// weights w is argmax_v w_v / e_v with e exponential: the race whose winner is v with probability w_v / sum
// w.  It needs no sum, so no order of summation can change a token.
//
// Only the row that the sequence draws from is read: p, q and e once, which HBM bounds for many sequences
// and the launches for few.  The vocabulary is split over workgroups; each finds the first unaccepted draft
// by itself (a few scalars) and leaves one key for each of the two draws (the rest, and p alone for the
// case that the rest is empty): the score's bits above the complement of the index, so that the largest key
// is the best score at the lowest index.  The second kernel takes the largest.
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
  uint64_t* keys;           // [batch][parts]
  int32_t* accepted;
  int32_t* out;             // [batch][drafts + 1]
  int32_t* err;
  int32_t batch, drafts, vocab, parts, per;  // per: entries of a part
};

// Workgroups that share out a row; 1: one of 1024 threads does it all in one launch (one compute unit alone
// draws no more than 40 GB/s: a row of 32000 takes it 14 us, 16 workgroups 5 us and the second launch 2).
inline int draft_parts(int32_t batch, int32_t vocab) {
  if (vocab <= 8192 || batch >= 512) return 1;
  // about 1024 workgroups in all, each of at least 2048 entries
  const int64_t most = ((int64_t)vocab + 2047) / 2048, want = (1024 + (batch > 0 ? batch : 1) - 1) / (batch > 0 ? batch : 1);
  return (int)(want < most ? want : most);
}

// Bytes of the parts' keys, of any smaller batch too: batch * parts < 1024 + batch where a row is shared out.
inline int64_t draft_keys_bytes(int32_t batch, int32_t vocab) {
  const int64_t whole = batch, shared = (int64_t)batch * draft_parts(1, vocab), most = 1023 + whole;
  return 8 * (shared < most ? shared : most);
}

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

// A draw's best so far: its score and index.  Entries come in ascending order of the index.
struct Best {
  float score = 0.0f;
  int at = -1;

  // Whether w / e may pass the score: at most one entry in a few hundred does, so the division is only
  // taken for those.  fl(w / e) > score needs w > score * e * (1 - 2^-24); the product's own rounding is
  // 2^-24 (not where it is subnormal: the test is passed there), and the factor below leaves room for both.
  __device__ __forceinline__ bool may(float w, float e) const {
    const float t = score * e;
    return w > 0.0f && e >= 0.0f && !(w < t * 0.999999f && t > 1e-30f);
  }
  __device__ __forceinline__ void take(float w, float e, int v) {
    const float s = __fdiv_rn(w, e);
    if (s > score || (at < 0 && s >= 0.0f)) score = s, at = v;
  }
  // bit 31 (a score has no sign) marks the key as one of a candidate
  __device__ __forceinline__ uint64_t key() const {
    return at < 0 ? 0 : (uint64_t)(__float_as_uint(score) | 0x80000000u) << 32 | (0xffffffffu - (uint32_t)at);
  }
};

__device__ __forceinline__ uint64_t wave_max(uint64_t k) {
#pragma unroll
  for (int d = 32; d; d >>= 1) {
    const uint64_t o = (uint64_t)__shfl_xor((unsigned long long)k, d);
    k = o > k ? o : k;
  }
  return k;
}

// A workgroup's best of entries [from, end) of the row that sequence b draws from, in every thread.
template <bool F32, int THREADS>
__device__ __forceinline__ uint64_t best_of(const DraftArgs& a, int b, int done, bool with_draft, int64_t from, int64_t end) {
  constexpr int kAhead = THREADS == 1024 ? 16 : 8;  // entries in flight a thread: one workgroup alone waits for each round of loads
  __shared__ uint64_t best[THREADS / 64];
  const int tid = threadIdx.x;
  const int n = a.counts ? min(max(a.counts[b], 0), a.drafts) : a.drafts;
  const bool less = with_draft && done < n;
  const int64_t row = ((int64_t)b * (a.drafts + 1) + done) * a.vocab;
  const int64_t qrow = ((int64_t)b * a.drafts + done) * a.vocab;
  const int certain = less && !a.draft ? a.tokens[(int64_t)b * a.drafts + done] : -1;
  const bool take = less && a.draft;
  const float* noise = a.noise + (int64_t)b * a.vocab;
  Best mine;
  for (int64_t v0 = from + tid; v0 < end; v0 += THREADS * kAhead) {
    float w[kAhead], e[kAhead], q[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int64_t v = v0 + THREADS * i;
      const bool in = v < end;
      w[i] = in ? prob<F32>(a.target, row + v) : 0.0f;
      e[i] = in ? noise[v] : 1.0f;
      q[i] = in && take ? prob<F32>(a.draft, qrow + v) : 0.0f;
    }
    bool any = false;
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      w[i] = (int)(v0 + THREADS * i) == certain ? 0.0f : w[i] - q[i];
      any |= mine.may(w[i], e[i]);
    }
    if (any) {
#pragma unroll
      for (int i = 0; i < kAhead; ++i)
        if (mine.may(w[i], e[i])) mine.take(w[i], e[i], (int)(v0 + THREADS * i));
    }
  }
  const uint64_t k = wave_max(mine.key());
  __syncthreads();  // (an earlier call's keys have been read)
  if ((tid & 63) == 0) best[tid >> 6] = k;
  __syncthreads();
  uint64_t top = best[0];
  for (int i = 1; i < THREADS / 64; ++i) top = best[i] > top ? best[i] : top;
  return top;
}

// The answer of sequence b, from the rest's best; where the rest was empty, from the target alone.
template <bool F32, int THREADS>
__device__ __forceinline__ void answer(const DraftArgs& a, int b, int done, bool bad, uint64_t k) {
  const int tid = threadIdx.x;
  if (k == 0) k = best_of<F32, THREADS>(a, b, done, false, 0, a.vocab);
  const int last = k ? (int)(0xffffffffu - (uint32_t)k) : -1;
  for (int i = tid; i <= a.drafts; i += THREADS)
    a.out[(int64_t)b * (a.drafts + 1) + i] = i < done ? a.tokens[(int64_t)b * a.drafts + i] : i == done ? last : -1;
  if (tid == 0) {
    a.accepted[b] = done;
    if (a.err && (bad || !k)) atomicAdd(a.err, 1);
  }
}

template <bool F32>
__global__ __launch_bounds__(1024) void k_draft_one(DraftArgs a) {
  const int b = blockIdx.x;
  bool bad;
  const int done = accepted_of<F32>(a, b, &bad);
  answer<F32, 1024>(a, b, done, bad, best_of<F32, 1024>(a, b, done, true, 0, a.vocab));
}

template <bool F32>
__global__ __launch_bounds__(256) void k_draft_part(DraftArgs a) {
  const int b = blockIdx.y;
  bool bad;
  const int done = accepted_of<F32>(a, b, &bad);
  const int64_t from = (int64_t)blockIdx.x * a.per;
  const uint64_t k = best_of<F32, 256>(a, b, done, true, from, min(from + a.per, (int64_t)a.vocab));
  if (threadIdx.x == 0) a.keys[(int64_t)b * a.parts + blockIdx.x] = k;
}

template <bool F32>
__global__ __launch_bounds__(256) void k_draft_pick(DraftArgs a) {
  const int b = blockIdx.x;
  bool bad;
  const int done = accepted_of<F32>(a, b, &bad);
  uint64_t k = 0;
  for (int i = threadIdx.x & 63; i < a.parts; i += 64) {
    const uint64_t x = a.keys[(int64_t)b * a.parts + i];
    k = x > k ? x : k;
  }
  answer<F32, 256>(a, b, done, bad, wave_max(k));  // (the same in every wave)
}

}  // namespace serve
