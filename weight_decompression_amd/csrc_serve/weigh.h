// The attention weight that cached tokens have received: for every key j of a sequence and key head,
//
//   w_j (+)= sum_i exp(scale q_i . k_j - lse_i)
//
// over the rows i (new tokens and query heads of the key head) that see it, lse_i the log-sum that the attention of the same
// rows gave.  With it a weight needs no other key: keys are shared out, rows are walked, nothing is split and joined, and
// no sum depends on an order of workgroups.
//
// S = Q K^T is taken with 32x32x16 bf16 instructions, rows down and keys across: a lane holds one key and 16 rows, so a
// key's sum is the lane's own (and its partner's, lane ^ 32).  A wave keeps its keys as operands in registers for the whole
// call, straight from memory, no LDS: which channels a step of the product takes does not matter as long as both operands
// agree, so a lane's 16 raw bytes (8, 16 or 32 channels) are one, two or four steps, and the rows are read from LDS in that
// order.  Scores, exponentials and sums are f32; f32 queries are three bf16 terms, as in attention.
//
// A decode step reads each key once for a handful of rows: HBM bounds it.  A chunk of a prompt walks thousands of rows over
// each key: the matrix instructions and the exponentials, a fused multiply-add, an exp and an add a score, share the time.
#pragma once

#include "attn.h"
#include "serve_common.h"

namespace serve {

struct WeighArgs {
  Cache c;
  const void* q;
  const float* lse;  // [tokens][heads]
  float* weights;    // [pages][heads][page]
  int64_t q_token, q_head;
  Divider share;
  int32_t tiles;     // workgroups of keys of a sequence; a longer one takes turns
  int32_t window, causal, fresh, max_rows, q_vec;
  float scale_log2;
  int32_t* err;
};

template <int DP, int NT>
struct WeighShape {
  static constexpr int kTiles = DP <= 128 ? 2 : 1;     // of 32 keys that a wave holds
  static constexpr int kKeys = 4 * 32 * kTiles;        // of a workgroup
  static constexpr int kRow = DP * 2 + 16;             // bytes of a row in LDS, padded as attention's keys are
};

// The channels of step st that lanes of `half` hold.
template <int KIND>
__device__ __forceinline__ constexpr int channel_of(int st, int half) {
  return KIND == LLVQ_KV_BF16 ? 16 * st + 8 * half : KIND == LLVQ_KV_FP8 ? 32 * (st / 2) + 16 * half + 8 * (st & 1) : 64 * (st / 4) + 32 * half + 8 * (st & 3);
}

template <int KIND, int DP, int NT>
__global__ __launch_bounds__(256, NT == 3 && DP == 256 ? 1 : 2) void k_weigh(WeighArgs a) {
  using Sh = WeighShape<DP, NT>;
  constexpr int kSteps = DP / 16, kTiles = Sh::kTiles;
  constexpr int kOf = KIND == LLVQ_KV_BF16 ? 1 : KIND == LLVQ_KV_FP8 ? 2 : 4;  // steps of a 16-byte chunk
  constexpr int kChunks = kSteps / kOf;                                        // chunks of a lane and key
  constexpr int kWords = KIND == LLVQ_KV_BF16 ? 1 : DP <= 128 ? 1 : 2;
  constexpr int kParts = 32 * (DP / 8) / 256;                                  // 8-channel parts of a row block a thread stages
  const Cache& c = a.c;
  __shared__ __align__(16) uint8_t rows_lds[2][NT][32 * Sh::kRow];
  __shared__ float lse_lds[2][32];
  __shared__ int pos_lds[2][32];  // a row's position, or far below any for none

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int half = lane >> 5, col = lane & 31;
  int id = blockIdx.x;
  const int head = id % c.heads;
  id /= c.heads;
  const int b = id / a.tiles, tile0 = id % a.tiles;
  const Seq s = sequence(c, b);
  const int share = (int)a.share.by, rows = min(s.n, a.max_rows) * share, text = s.len - s.n, heads = c.heads * share;
  if (a.err && tid == 0 && head == 0 && tile0 == 0 && (s.bad || s.n > a.max_rows)) atomicAdd(a.err, 1);
  if (s.n == 0) return;
  const int32_t* table = c.table + (int64_t)b * c.max_pages;
  bool lost = false;

  for (int tile = tile0; (int64_t)tile * Sh::kKeys < s.len; tile += a.tiles) {
    const int key0 = tile * Sh::kKeys + wave * 32 * kTiles;
    // the rows that see any key of the workgroup's: tokens [t0, t1)
    const int first_key = tile * Sh::kKeys, last_key = min(first_key + Sh::kKeys, s.len) - 1;
    const int t0 = a.causal ? max(first_key - text, 0) : 0;
    const int64_t reach = (int64_t)last_key - text + a.window;
    const int t1 = a.window > 0 ? (int)min((int64_t)min(s.n, a.max_rows), max(reach, (int64_t)0)) : min(s.n, a.max_rows);
    const int block0 = t0 * share / 32, block1 = t1 > t0 ? (t1 * share + 31) / 32 : block0;

    // the keys
    float* at[kTiles];
    bf16x8 k[kTiles][kSteps];
    float sum[kTiles];
#pragma unroll
    for (int u = 0; u < kTiles; ++u) {
      const int j = key0 + u * 32 + col;
      const uint32_t page = divide((uint32_t)j, c.page);
      const int32_t pid = j < s.len ? table[page] : -1;
      const bool ok = pid >= 0 && pid < c.pages;
      lost |= j < s.len && !ok;
      const int slot = j - (int)(page * c.page.by);
      at[u] = ok ? a.weights + ((int64_t)pid * c.heads + head) * c.page.by + slot : nullptr;
      const uint8_t* blk = c.pool + (ok ? ((int64_t)pid * c.heads + head) * c.block : 0);
      const uint8_t* row = blk + (ok ? slot * c.row : 0);
      u32x4 raw[kChunks];
      uint32_t words[kWords];
#pragma unroll
      for (int m = 0; m < kChunks; ++m) {
        const int ch = 2 * m + half;
        raw[m] = u32x4{0, 0, 0, 0};
        if (ok && ch * 16 < c.row) raw[m] = *reinterpret_cast<const u32x4*>(row + ch * 16);
      }
#pragma unroll
      for (int n = 0; n < kWords; ++n) {
        words[n] = 0x7f7f7f7fu;
        if (KIND != LLVQ_KV_BF16 && ok) words[n] = scale_word(blk + c.ks_off + slot * c.groups, c.groups, n);
      }
      nan_scales<KIND, kWords>(words);
#pragma unroll
      for (int m = 0; m < kChunks; ++m) {
        const int group = channel_of<KIND>(m * kOf, half) / 32;
        const uint32_t sb = KIND == LLVQ_KV_BF16 ? 127 : words[group / 4 % kWords] >> (8 * (group % 4)) & 255;
        u32x4 o[kOf];
        expand<KIND>(raw[m], sb, o);
#pragma unroll
        for (int e = 0; e < kOf; ++e) k[u][m * kOf + e] = __builtin_bit_cast(bf16x8, o[e]);
      }
      sum[u] = 0.0f;
    }

    // a block of rows into LDS
    auto stage = [&](int block, int buffer) {
#pragma unroll
      for (int i = 0; i < kParts; ++i) {
        const int part = i * 256 + tid, r = part / (DP / 8), ch = part % (DP / 8) * 8;
        const int row = block * 32 + r;
        const bool live = row < rows;
        const int t = live ? (int)divide((uint32_t)row, a.share) : 0;
        const int64_t from = (int64_t)(s.first + t) * a.q_token + (int64_t)(head * share + (live ? row - t * share : 0)) * a.q_head;
        float x[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = 0.0f;
        if (live && ch < c.dim) {
          if (a.q_vec)
            load8<NT == 3, true>(a.q, from + ch, x);
          else
            load8<NT == 3, false>(a.q, from + ch, x);
        }
        bf16x8 terms[NT];
        split_terms<NT>(x, terms);
#pragma unroll
        for (int n = 0; n < NT; ++n) *reinterpret_cast<bf16x8*>(&rows_lds[buffer][n][r * Sh::kRow + ch * 2]) = terms[n];
      }
      if (tid < 32) {
        const int row = block * 32 + tid;
        const bool live = row < rows;
        const int t = live ? (int)divide((uint32_t)row, a.share) : 0;
        const float l = live ? a.lse[(int64_t)(s.first + t) * heads + head * share + (row - t * share)] : 0.0f;
        lse_lds[buffer][tid] = l * 1.4426950408889634f;
        pos_lds[buffer][tid] = live ? text + t : -0x7fffffff;
      }
    };

    __syncthreads();  // (the tile before has been worked through)
    if (block0 < block1) stage(block0, 0);
    for (int block = block0; block < block1; ++block) {
      const int buffer = (block - block0) & 1;
      __syncthreads();
      if (block + 1 < block1) stage(block + 1, buffer ^ 1);
      const int p0 = pos_lds[buffer][0], p1 = pos_lds[buffer][31];
      // whether every row sees every key of the wave's
      const int hi = key0 + 32 * kTiles - 1;
      const bool whole = p1 >= text && (!a.causal || hi <= p0) && (a.window == 0 || key0 > p1 - a.window);
#pragma unroll
      for (int u = 0; u < kTiles; ++u) {
        f32x16 sc = {0.0f};
#pragma unroll
        for (int st = 0; st < kSteps; ++st)
#pragma unroll
          for (int n = NT - 1; n >= 0; --n) {
            const bf16x8 qf = *reinterpret_cast<const bf16x8*>(&rows_lds[buffer][n][col * Sh::kRow + channel_of<KIND>(st, half) * 2]);
            sc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(qf, k[u][st], sc, 0, 0, 0);
          }
        float part[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        const int j = key0 + u * 32 + col;
#pragma unroll
        for (int i4 = 0; i4 < 4; ++i4) {
          const f32x4 l = *reinterpret_cast<const f32x4*>(&lse_lds[buffer][i4 * 8 + half * 4]);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            float p = __builtin_amdgcn_exp2f(fmaf(sc[i4 * 4 + i], a.scale_log2, -l[i]));
            if (!whole) {
              const int pos = pos_lds[buffer][i4 * 8 + half * 4 + i];
              const bool see = pos != -0x7fffffff && (!a.causal || j <= pos) && (a.window == 0 || j > pos - a.window);
              p = see ? p : 0.0f;
            }
            part[i] += p;
          }
        }
        sum[u] += (part[0] + part[1]) + (part[2] + part[3]);
      }
    }
    // what the new tokens' places held is of earlier tokens
#pragma unroll
    for (int u = 0; u < kTiles; ++u) {
      const float got = half_sum(sum[u]);
      const int j = key0 + u * 32 + col;
      if (half == 0 && at[u]) *at[u] = (a.fresh || j >= text ? 0.0f : *at[u]) + got;
    }
  }
  if (a.err && lost) atomicAdd(a.err, 1);
}

}  // namespace serve
