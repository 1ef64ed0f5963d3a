// Host side of attention over the paged cache: the rules that cut a call into workgroups, its checks and launches,
// for the units that hold its forms (plain, trees, with the rows' log-sums).
#pragma once

#include <math.h>

#include "attn.h"
#include "serve_host.h"

namespace serve {
namespace {

// How a call is cut up: columns of 16 that a team of the kernel for few rows holds (0: the kernel for many rows), waves
// of a team (or of a workgroup of the other kernel), row blocks and splits of the keys.
struct Cut {
  int cols, waves, row_blocks, splits;
};

inline int padded_dim(int dim) { return dim <= 64 ? 64 : dim <= 128 ? 128 : 256; }

// The rules go by sizes that the host knows; times are of whole calls on one MI355X.
// A window only makes the splits fewer.
inline int cut_of(const llvq_kv_desc* d, int64_t share, int32_t batch, int32_t max_chunk, int32_t max_len, int32_t window, bool f32,
           Cut* cut) {
  if (window > 0 && max_len - max_chunk > window) max_len = window + max_chunk;
  const int64_t rows = (int64_t)max_chunk * share, seqs = (int64_t)d->kv_heads * (batch > 0 ? batch : 1);
  const int dim = padded_dim(d->head_dim), parts = dim > 128 ? 2 : 1, terms = f32 ? 3 : 1;
  if (rows * seqs > (1ll << 33)) return LLVQ_EINVAL;
  cut->waves = 4;
  cut->cols = rows > 64 ? 0 : rows <= 16 || !few_pairs(d->kind, dim, terms) ? 1 : 2;
  // Eight waves stage a tile for 256 rows: 478 us instead of 530 at chunks of 2 x 2048 of 32 128-wide heads
  // over 8192 keys, 196 instead of 218 at 256-wide heads.  64-wide heads run better with three workgroups
  // of four a compute unit (87 us, 113 with eight waves), and where 256 rows a workgroup leave compute
  // units idle, 128 do better (369 rows of 32 heads: 17 us instead of 19)
  if (!cut->cols && !f32 && dim > 64 && rows > 128 && (rows + 255) / 256 * seqs * parts >= 256) cut->waves = 8;
  const int64_t per = cut->cols ? 16 * cut->cols : 32 * cut->waves;
  const int64_t blocks = (rows + per - 1) / per, base = blocks * seqs;
  if (base > (1ll << 29)) return LLVQ_EINVAL;
  int64_t s;
  if (cut->cols) {
    // Up to half a chip's workgroups: as many parts as fill one round of resident ones (three sequences of 131000
    // keys in e2m1: 81 us at 768 workgroups, 93 at 2048).  Twice a chip: no split (57 x 32 of up to 176 keys: 54
    // us, 72 split).  Between, a split fills what the last round leaves idle and evens out lengths, and costs its
    // sums' way out and back: it needs long sequences, and longer ones where one round is nearly full.  Times split
    // over unsplit, geometric means of equal and of ragged lengths (a quarter of max_len on) and of bf16 and f32
    // queries with own and shared keys, 128-wide heads in e4m3, at workgroups over resident ones of
    //             0.55  0.65  0.75  0.85  1.0   1.2   1.5
    //   2000 keys 1.18  1.19  1.16  1.22  1.32  1.09  1.15
    //   3000      1.05  1.04  1.07  1.14  1.22  0.99  1.07
    //   4096      0.99  1.02  1.02  1.09  1.16  0.97  1.06
    //   6000      0.92  1.01  0.97  1.07  1.11  0.92  1.00
    //   8192      0.87  0.97  0.99  1.00  1.07  0.88  1.00
    // bf16 at 4096 0.90 to 1.04, e2m1 0.91 to 1.11, 64-wide bf16 0.93 to 1.03, 256-wide e4m3 0.97 to 1.40.  The means
    // hide the lengths' spread: 424 e4m3 workgroups of 4096 keys, 0.91 ragged and 1.19 equal.
    const int64_t resident = 256 * few_waves(d->kind, dim, terms, cut->cols);
    const bool full = base > resident * 4 / 5 && base <= resident;
    s = base <= resident / 2                                      ? resident / base
        : base >= 2 * resident || max_len <= (full ? 8192 : 4096) ? 1
                                                                  : (2048 + base - 1) / base;
    const int64_t most = ((int64_t)max_len + 127) / 128;
    if (s > most) s = most;
    // Short sequences that fill the chip a wave each (64 x 32 in e4m3 of up to 500 keys: 39 us, 42 with four
    // waves; of up to 1000 78 and 73)
    if (base >= 2 * resident && max_len <= 768) cut->waves = 1;
    // Eight waves a workgroup and no split, so one launch: 5 us and about 2.1 more for each 256 keys, while a split
    // call of few workgroups takes 10 us on the device and 13 in a stream of calls.  Up to 64 workgroups the one launch
    // pays up to 768 keys (8 x 4 heads of shared keys in e4m3: of 768 keys 11.4 us, split 10.1, in a stream 11.8 and
    // 13.5; of 896 13.6 and 10.3, in a stream 14.0 and 13.1; bf16, e2m1 and f32 queries alike).  More workgroups leave a
    // split less to fill.  Split over one launch: 128 workgroups of 1024 keys 0.93 to 1.11, 1280 0.90 to 1.23, 1536
    // 0.87 to 1.12; 192 of 2048 0.91 to 1.16, 2560 0.95 to 1.13; 256 of 2560 1.02 to 1.12.
    const int64_t one_launch = 10 * base > 768 ? 10 * base : 768;
    if (cut->cols == 1 && dim <= 128 && base <= 256 && max_len <= one_launch) cut->waves = 8, s = 1;
  } else {
    // A split shortens a workgroup's way (about 1 us a tile of 64 keys; f32 and wide heads more) and costs
    // its sums' way out and back (8 bytes a channel of every row at 5 TB/s): the least of tiles / s + cost
    // * s, up to two rounds of workgroups (3 x 295 rows of 12 heads in a window of 1932 keys: 37 us at 6
    // splits, 56 at 12)
    const int64_t slots = 256 * (cut->waves == 8 ? 1 : dim == 64 && !f32 ? 3 : 2);
    const double tiles = max_len / 64.0 * (f32 ? 2.5 : 1.0) * parts, cost = (double)rows * seqs * d->head_dim * 8.0 / 5e6;
    s = (2 * slots + base * parts / 2) / (base * parts);
    const int64_t best = (int64_t)sqrt(tiles / cost), most = ((int64_t)max_len + 127) / 128;
    if (s > best) s = best;
    if (s > most) s = most;
  }
  cut->splits = (int)(s < 1 ? 1 : s > kMaxSplits ? kMaxSplits : s);
  cut->row_blocks = (int)blocks;
  // (a launch has fewer than 2^32 threads)
  return base * cut->splits * parts * 64 * cut->waves >= (1ll << 32) ? LLVQ_EINVAL : LLVQ_OK;
}

// The sums, maxima and sums of p of that many (row, split) pairs.
inline int64_t workspace_of(const llvq_kv_desc* d, int64_t rows) { return rows * (d->head_dim + 2) * 4; }

// (row, split) pairs that no split call passes.  Few rows: a call of base workgroups is split into resident / base or
// ceil(2048 / base) parts, so into fewer than 4096 workgroups, of up to 32 rows.  Many: into s >= 2 parts of base *
// parts * (s - 1/2) <= 2 slots, so into at most 8/3 slots workgroups, of 128 or 256 rows, 2^16 (64-wide heads: 3 *
// 2^15) on all slots.
inline int64_t most_split_rows(int head_dim) {
  const int dim = padded_dim(head_dim);
  const int64_t few = 4096 * 32, many = (dim == 64 ? 3ll << 15 : 1ll << 16) * 8 / 3 / (dim > 128 ? 2 : 1);
  return few > many ? few : many;
}

inline int check_attn(const llvq_kv_desc* d, int32_t heads, int64_t tokens, int32_t batch, int32_t max_chunk, int32_t max_len) {
  const int st = check_desc(d);
  if (st != LLVQ_OK) return st;
  if (heads < d->kv_heads || heads % d->kv_heads || heads > 65536) return LLVQ_EINVAL;
  if (tokens < 0 || tokens * heads > 0x7fffffff || batch < 0 || batch > LLVQ_MAX_SEQS) return LLVQ_EINVAL;
  if (tokens > (int64_t)batch * max_chunk) return LLVQ_EINVAL;
  if (max_chunk < 1 || max_len < 1 || max_len > kMaxLen || (int64_t)max_chunk * heads > 0x7fffffff) return LLVQ_EINVAL;
  return LLVQ_OK;
}

template <int MODE, int KIND, int DP, int NT, int WAVES>
int launch_many(const AttnArgs& a, unsigned grid, hipStream_t s) {
  using Sh = ManyShape<KIND, DP, NT, WAVES>;
  hipLaunchKernelGGL((k_attn_many<KIND, DP, NT, WAVES, MODE>), dim3(grid * Sh::kParts), dim3(Sh::kThreads), 0, s, a);
  return launch_status();
}
template <int MODE, int KIND, int DP, int NT, int CT, int TEAM>
int launch_few(const AttnArgs& a, unsigned grid, hipStream_t s) {
  hipLaunchKernelGGL((k_attn_few<KIND, DP, NT, CT, TEAM, MODE>), dim3(TEAM == 1 ? (grid + 3) / 4 : grid), dim3(TEAM == 8 ? 512 : 256), 0, s, a);
  return launch_status();
}
template <int MODE, int KIND, int DP, int NT>
int launch_attn(const AttnArgs& a, const Cut& cut, unsigned grid, hipStream_t s) {
  if constexpr (NT == 1 && DP > 64) {
    if (cut.cols == 0 && cut.waves == 8) return launch_many<MODE, KIND, DP, NT, 8>(a, grid, s);
  }
  if (cut.cols == 0) return launch_many<MODE, KIND, DP, NT, 4>(a, grid, s);
  if constexpr (few_pairs(KIND, DP, NT)) {
    if (cut.cols == 2)
      return cut.waves == 1 ? launch_few<MODE, KIND, DP, NT, 2, 1>(a, grid, s) : launch_few<MODE, KIND, DP, NT, 2, 4>(a, grid, s);
  }
  if (cut.waves == 1) return launch_few<MODE, KIND, DP, NT, 1, 1>(a, grid, s);
  if constexpr (DP <= 128) {
    if (cut.waves == 8) return launch_few<MODE, KIND, DP, NT, 1, 8>(a, grid, s);
  }
  return launch_few<MODE, KIND, DP, NT, 1, 4>(a, grid, s);
}
template <int MODE, int KIND, int DP>
int launch_attn_nt(const AttnArgs& a, bool f32, const Cut& cut, unsigned grid, hipStream_t s) {
  return f32 ? launch_attn<MODE, KIND, DP, 3>(a, cut, grid, s) : launch_attn<MODE, KIND, DP, 1>(a, cut, grid, s);
}
template <int MODE, int KIND>
int launch_attn_dp(const AttnArgs& a, bool f32, const Cut& cut, unsigned grid, hipStream_t s) {
  switch (padded_dim(a.c.dim)) {
    case 64: return launch_attn_nt<MODE, KIND, 64>(a, f32, cut, grid, s);
    case 128: return launch_attn_nt<MODE, KIND, 128>(a, f32, cut, grid, s);
    default: return launch_attn_nt<MODE, KIND, 256>(a, f32, cut, grid, s);
  }
}

template <int MODE, bool F32, int LANES>
int launch_join(const AttnArgs& a, hipStream_t s) {
  const int64_t rows = (int64_t)a.c.tokens * a.c.heads * a.share.by;
  // Four waves a row from 8 splits on: 96 rows of 86 splits of 128 channels take 7.5 us, one wave a row 47 us
  if (a.splits >= 8)
    hipLaunchKernelGGL((k_attn_join<F32, LANES, 4, MODE>), dim3((unsigned)rows), dim3(256), 0, s, a);
  else
    hipLaunchKernelGGL((k_attn_join<F32, LANES, 1, MODE>), dim3((unsigned)((rows + 3) / 4)), dim3(256), 0, s, a);
  return launch_status();
}
template <int MODE, bool F32>
int launch_join_dim(const AttnArgs& a, hipStream_t s) {
  switch (padded_dim(a.c.dim)) {
    case 64: return launch_join<MODE, F32, 16>(a, s);
    case 128: return launch_join<MODE, F32, 32>(a, s);
    default: return launch_join<MODE, F32, 64>(a, s);
  }
}

// llvq_attn and its forms: parents only for trees (kTree), lse only for kLse.
template <int MODE>
int attn_call(const llvq_kv_desc* d, const void* pool, const void* q, int64_t q_token, int64_t q_head, void* out,
              int64_t out_token, int64_t out_head, int32_t dtype, int32_t heads, const llvq_batch* batch,
              const int32_t* parents, int32_t max_chunk, int32_t max_len, float scale, int32_t causal, int32_t window, float* lse,
              void* workspace, int64_t workspace_bytes, int32_t* err_count, void* stream) {
  Cache c;
  int st = make_cache(d, pool, batch, &c);
  if (st != LLVQ_OK) return st;
  st = check_attn(d, heads, batch->tokens, batch->batch, max_chunk, max_len);
  if (st != LLVQ_OK) return st;
  if (dtype != LLVQ_X_F32 && dtype != LLVQ_X_BF16) return LLVQ_EINVAL;
  const float scale_log2 = (float)((double)scale * 1.4426950408889634);
  if (!(scale > 0.0f) || !(scale_log2 < INFINITY) || window < 0 || window > kMaxLen) return LLVQ_EINVAL;
  if (err_count && !aligned(err_count, 4)) return LLVQ_EINVAL;
  if (MODE == kTree && max_chunk > LLVQ_MAX_NODES) return LLVQ_EINVAL;
  if (c.tokens == 0 || c.batch == 0) return LLVQ_OK;
  if (MODE == kTree && (!parents || !aligned(parents, 4))) return LLVQ_EINVAL;
  if (MODE == kLse && (!lse || !aligned(lse, 4))) return LLVQ_EINVAL;
  const bool f32 = dtype == LLVQ_X_F32;
  const int size = f32 ? 4 : 2;
  if (!q || !out || !aligned(q, size) || !aligned(out, 4 * size)) return LLVQ_EINVAL;
  if (q_token < 0 || q_head < 0 || out_token < 0 || out_head < 0 || out_token % 4 || out_head % 4) return LLVQ_EINVAL;
  Cut cut;
  st = cut_of(d, heads / d->kv_heads, c.batch, max_chunk, max_len, window, f32, &cut);
  if (st != LLVQ_OK) return st;
  const int64_t need = cut.splits > 1 ? workspace_of(d, (int64_t)cut.splits * c.tokens * heads) : 0;
  if (need > 0 && (!workspace || !aligned(workspace, 16) || workspace_bytes < need)) return LLVQ_EINVAL;
  AttnArgs a = {};
  a.c = c;
  a.q = q;
  a.out = out;
  a.q_token = q_token;
  a.q_head = q_head;
  a.out_token = out_token;
  a.out_head = out_head;
  a.share = make_divider((uint32_t)(heads / d->kv_heads));
  a.row_blocks = cut.row_blocks;
  a.splits = cut.splits;
  a.window = window;
  a.causal = causal != 0;
  a.q_vec = wide(q, q_token, q_head, size);
  a.scale_log2 = scale_log2;
  a.err = err_count;
  a.parents = parents;
  a.lse = lse;
  if (cut.splits > 1) {
    a.part = static_cast<float*>(workspace);
    a.stats = a.part + (int64_t)cut.splits * c.tokens * heads * c.dim;
  }
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  const unsigned grid = (unsigned)((int64_t)c.batch * cut.row_blocks * cut.splits * c.heads);
  a.units = (int32_t)grid;
  switch (d->kind) {
    case LLVQ_KV_BF16: st = launch_attn_dp<MODE, LLVQ_KV_BF16>(a, f32, cut, grid, s); break;
    case LLVQ_KV_FP8: st = launch_attn_dp<MODE, LLVQ_KV_FP8>(a, f32, cut, grid, s); break;
    default: st = launch_attn_dp<MODE, LLVQ_KV_FP4>(a, f32, cut, grid, s); break;
  }
  if (st != LLVQ_OK || cut.splits == 1) return st;
  return f32 ? launch_join_dim<MODE, true>(a, s) : launch_join_dim<MODE, false>(a, s);
}

}  // namespace
}  // namespace serve
