// Host side of the serving calls of include/llvq.h: the paged key/value cache, the attention over it
// and the check of drafted tokens.  Arguments are validated here, before any launch; kernels bound every
// index that they read from device memory by what the host was told.
#include <math.h>

#include "attn.h"
#include "draft.h"
#include "kv_cache.h"
#include "serve_common.h"

#define LLVQ_API extern "C" __attribute__((visibility("default")))

using namespace serve;

namespace {

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
int launch_status() { return hipGetLastError() == hipSuccess ? LLVQ_OK : LLVQ_EHIP; }

int64_t block_bytes(const llvq_kv_desc* d) {
  const int64_t groups = d->kind == LLVQ_KV_BF16 ? 0 : d->head_dim / kGroup;
  return (2 * d->page_tokens * (code_bytes(d->kind, d->head_dim) + groups) + 15) / 16 * 16;
}

int check_desc(const llvq_kv_desc* d) {
  if (!d || d->kind < LLVQ_KV_BF16 || d->kind > LLVQ_KV_FP4) return LLVQ_EINVAL;
  if (d->kv_heads < 1 || d->kv_heads > 1024 || d->pages < 1) return LLVQ_EINVAL;
  if (d->head_dim < kGroup || d->head_dim > LLVQ_MAX_HEAD_DIM || d->head_dim % kGroup) return LLVQ_EINVAL;
  if (d->page_tokens < 1 || d->page_tokens > LLVQ_MAX_PAGE) return LLVQ_EINVAL;
  return LLVQ_OK;
}

int make_cache(const llvq_kv_desc* d, const void* pool, const llvq_batch* n, Cache* c) {
  const int st = check_desc(d);
  if (st != LLVQ_OK) return st;
  if (!n || n->batch < 0 || n->batch > LLVQ_MAX_SEQS || n->tokens < 0 || n->tokens > LLVQ_MAX_TOKENS || n->max_pages < 0) return LLVQ_EINVAL;
  if (n->batch > 0 && n->tokens > 0) {
    if (!pool || !n->starts || !n->lens || (n->max_pages > 0 && !n->table)) return LLVQ_EINVAL;
    if (!aligned(pool, 16) || !aligned(n->starts, 4) || !aligned(n->lens, 4) || !aligned(n->table, 4)) return LLVQ_EINVAL;
  }
  *c = Cache{};
  c->pool = static_cast<uint8_t*>(const_cast<void*>(pool));
  c->starts = n->starts;
  c->lens = n->lens;
  c->table = n->table;
  c->block = block_bytes(d);
  c->page = make_divider((uint32_t)d->page_tokens);
  c->heads = d->kv_heads;
  c->dim = d->head_dim;
  c->pages = d->pages;
  c->batch = n->batch;
  c->max_pages = n->max_pages;
  c->tokens = n->tokens;
  c->row = code_bytes(d->kind, d->head_dim);
  c->groups = d->kind == LLVQ_KV_BF16 ? 0 : d->head_dim / kGroup;
  c->v_off = d->page_tokens * c->row;
  c->ks_off = 2 * c->v_off;
  c->vs_off = c->ks_off + d->page_tokens * c->groups;
  return LLVQ_OK;
}

// Whether rows of `bytes`-wide elements can be moved 16 bytes at a time.
bool wide(const void* p, int64_t token, int64_t head, int bytes) {
  return aligned(p, 16) && (token * bytes) % 16 == 0 && (head * bytes) % 16 == 0;
}

template <int KIND, bool WRITE, int PW>
int launch_kv(const Cache& c, const KvRows& r, bool f32, bool vec, int32_t* err, hipStream_t s) {
  const int items = 2 * c.heads * (c.dim / 8);
  const Divider chunks = make_divider((uint32_t)(c.dim / 8));
  const unsigned gx = (unsigned)((c.tokens + 4ll * PW - 1) / (4ll * PW));
  const unsigned parts = (unsigned)((items + kWave - 1) / kWave);
  // a wave has one item of each token while that leaves it few workgroups, up to four after that
  const unsigned gy = (uint64_t)gx * parts >= 1024 ? (parts + 3) / 4 : parts;
  const dim3 grid(gx, gy > 65535 ? 65535 : gy);
#define LLVQ_KV_CASE(F32, VEC)                                                                                \
  if (f32 == F32 && vec == VEC) {                                                                             \
    if constexpr (WRITE)                                                                                      \
      hipLaunchKernelGGL((k_kv_write<KIND, F32, VEC, PW>), grid, dim3(256), 0, s, c, r, chunks, items, err);  \
    else                                                                                                      \
      hipLaunchKernelGGL((k_kv_read<KIND, F32, VEC, PW>), grid, dim3(256), 0, s, c, r, chunks, items, err);   \
  }
  LLVQ_KV_CASE(false, false) LLVQ_KV_CASE(false, true) LLVQ_KV_CASE(true, false) LLVQ_KV_CASE(true, true)
#undef LLVQ_KV_CASE
  return launch_status();
}

template <bool WRITE>
int kv_call(const llvq_kv_desc* d, const void* pool, const void* k, int64_t k_token, int64_t k_head, const void* v,
            int64_t v_token, int64_t v_head, int32_t dtype, const llvq_batch* n, int32_t* err, void* stream) {
  Cache c;
  const int st = make_cache(d, pool, n, &c);
  if (st != LLVQ_OK) return st;
  if (dtype != LLVQ_X_F32 && dtype != LLVQ_X_BF16) return LLVQ_EINVAL;
  if (err && !aligned(err, 4)) return LLVQ_EINVAL;
  if (c.tokens == 0 || c.batch == 0) return LLVQ_OK;
  const bool f32 = dtype == LLVQ_X_F32;
  const int size = f32 ? 4 : 2;
  if (!k || !v || !aligned(k, size) || !aligned(v, size)) return LLVQ_EINVAL;
  if (k_token < 0 || k_head < 0 || v_token < 0 || v_head < 0) return LLVQ_EINVAL;
  const bool vec = wide(k, k_token, k_head, size) && wide(v, v_token, v_head, size);
  const KvRows r = {k, v, k_token, k_head, v_token, v_head};
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  // Four tokens a wave once that fills the chip: four loads in flight, and neighbours of a page written
  // together
  const bool four = (int64_t)c.tokens * c.heads * c.dim >= 1 << 22;
#define LLVQ_KV_KIND(KIND) four ? launch_kv<KIND, WRITE, 4>(c, r, f32, vec, err, s) : launch_kv<KIND, WRITE, 1>(c, r, f32, vec, err, s)
  switch (d->kind) {
    case LLVQ_KV_BF16: return LLVQ_KV_KIND(LLVQ_KV_BF16);
    case LLVQ_KV_FP8: return LLVQ_KV_KIND(LLVQ_KV_FP8);
    default: return LLVQ_KV_KIND(LLVQ_KV_FP4);
  }
#undef LLVQ_KV_KIND
}

// How a call is cut up: columns of 16 that a team of the kernel for few rows holds (0: the kernel for many rows), waves
// of a team (or of a workgroup of the other kernel), row blocks and splits of the keys.
struct Cut {
  int cols, waves, row_blocks, splits;
};

int padded_dim(int dim) { return dim <= 64 ? 64 : dim <= 128 ? 128 : 256; }

// The rules go by sizes that the host knows; times are of whole calls on one MI355X.
// A window only makes the splits fewer.
int cut_of(const llvq_kv_desc* d, int64_t share, int32_t batch, int32_t max_chunk, int32_t max_len, int32_t window, bool f32,
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
int64_t workspace_of(const llvq_kv_desc* d, int64_t rows) { return rows * (d->head_dim + 2) * 4; }

// (row, split) pairs that no split call passes.  Few rows: a call of base workgroups is split into resident / base or
// ceil(2048 / base) parts, so into fewer than 4096 workgroups, of up to 32 rows.  Many: into s >= 2 parts of base *
// parts * (s - 1/2) <= 2 slots, so into at most 8/3 slots workgroups, of 128 or 256 rows, 2^16 (64-wide heads: 3 *
// 2^15) on all slots.
int64_t most_split_rows(int head_dim) {
  const int dim = padded_dim(head_dim);
  const int64_t few = 4096 * 32, many = (dim == 64 ? 3ll << 15 : 1ll << 16) * 8 / 3 / (dim > 128 ? 2 : 1);
  return few > many ? few : many;
}

int check_attn(const llvq_kv_desc* d, int32_t heads, int64_t tokens, int32_t batch, int32_t max_chunk, int32_t max_len) {
  const int st = check_desc(d);
  if (st != LLVQ_OK) return st;
  if (heads < d->kv_heads || heads % d->kv_heads || heads > 65536) return LLVQ_EINVAL;
  if (tokens < 0 || tokens * heads > 0x7fffffff || batch < 0 || batch > LLVQ_MAX_SEQS) return LLVQ_EINVAL;
  if (tokens > (int64_t)batch * max_chunk) return LLVQ_EINVAL;
  if (max_chunk < 1 || max_len < 1 || max_len > kMaxLen || (int64_t)max_chunk * heads > 0x7fffffff) return LLVQ_EINVAL;
  return LLVQ_OK;
}

template <int KIND, int DP, int NT, int WAVES>
int launch_many(const AttnArgs& a, unsigned grid, hipStream_t s) {
  using Sh = ManyShape<KIND, DP, NT, WAVES>;
  hipLaunchKernelGGL((k_attn_many<KIND, DP, NT, WAVES>), dim3(grid * Sh::kParts), dim3(Sh::kThreads), 0, s, a);
  return launch_status();
}
template <int KIND, int DP, int NT, int CT, int TEAM>
int launch_few(const AttnArgs& a, unsigned grid, hipStream_t s) {
  hipLaunchKernelGGL((k_attn_few<KIND, DP, NT, CT, TEAM>), dim3(TEAM == 1 ? (grid + 3) / 4 : grid), dim3(TEAM == 8 ? 512 : 256), 0, s, a);
  return launch_status();
}
template <int KIND, int DP, int NT>
int launch_attn(const AttnArgs& a, const Cut& cut, unsigned grid, hipStream_t s) {
  if constexpr (NT == 1 && DP > 64) {
    if (cut.cols == 0 && cut.waves == 8) return launch_many<KIND, DP, NT, 8>(a, grid, s);
  }
  if (cut.cols == 0) return launch_many<KIND, DP, NT, 4>(a, grid, s);
  if constexpr (few_pairs(KIND, DP, NT)) {
    if (cut.cols == 2)
      return cut.waves == 1 ? launch_few<KIND, DP, NT, 2, 1>(a, grid, s) : launch_few<KIND, DP, NT, 2, 4>(a, grid, s);
  }
  if (cut.waves == 1) return launch_few<KIND, DP, NT, 1, 1>(a, grid, s);
  if constexpr (DP <= 128) {
    if (cut.waves == 8) return launch_few<KIND, DP, NT, 1, 8>(a, grid, s);
  }
  return launch_few<KIND, DP, NT, 1, 4>(a, grid, s);
}
template <int KIND, int DP>
int launch_attn_nt(const AttnArgs& a, bool f32, const Cut& cut, unsigned grid, hipStream_t s) {
  return f32 ? launch_attn<KIND, DP, 3>(a, cut, grid, s) : launch_attn<KIND, DP, 1>(a, cut, grid, s);
}
template <int KIND>
int launch_attn_dp(const AttnArgs& a, bool f32, const Cut& cut, unsigned grid, hipStream_t s) {
  switch (padded_dim(a.c.dim)) {
    case 64: return launch_attn_nt<KIND, 64>(a, f32, cut, grid, s);
    case 128: return launch_attn_nt<KIND, 128>(a, f32, cut, grid, s);
    default: return launch_attn_nt<KIND, 256>(a, f32, cut, grid, s);
  }
}

template <bool F32, int LANES>
int launch_join(const AttnArgs& a, hipStream_t s) {
  const int64_t rows = (int64_t)a.c.tokens * a.c.heads * a.share.by;
  // Four waves a row from 8 splits on: 96 rows of 86 splits of 128 channels take 7.5 us, one wave a row 47 us
  if (a.splits >= 8)
    hipLaunchKernelGGL((k_attn_join<F32, LANES, 4>), dim3((unsigned)rows), dim3(256), 0, s, a);
  else
    hipLaunchKernelGGL((k_attn_join<F32, LANES, 1>), dim3((unsigned)((rows + 3) / 4)), dim3(256), 0, s, a);
  return launch_status();
}
template <bool F32>
int launch_join_dim(const AttnArgs& a, hipStream_t s) {
  switch (padded_dim(a.c.dim)) {
    case 64: return launch_join<F32, 16>(a, s);
    case 128: return launch_join<F32, 32>(a, s);
    default: return launch_join<F32, 64>(a, s);
  }
}

// Workgroups that share out a row; 1: one of 1024 threads does it all in one launch (one compute unit alone
// draws no more than 40 GB/s: a row of 32000 takes it 14 us, 16 workgroups 5 us and the second launch 2).
int draft_parts(int32_t batch, int32_t vocab) {
  if (vocab <= 8192 || batch >= 512) return 1;
  // about 1024 workgroups in all, each of at least 2048 entries
  const int64_t most = ((int64_t)vocab + 2047) / 2048, want = (1024 + (batch > 0 ? batch : 1) - 1) / (batch > 0 ? batch : 1);
  return (int)(want < most ? want : most);
}

template <bool F32>
int launch_draft(const DraftArgs& a, hipStream_t s) {
  if (a.parts == 1) {
    hipLaunchKernelGGL((k_draft_one<F32>), dim3(a.batch), dim3(1024), 0, s, a);
  } else {
    hipLaunchKernelGGL((k_draft_part<F32>), dim3(a.parts, a.batch), dim3(256), 0, s, a);
    hipLaunchKernelGGL((k_draft_pick<F32>), dim3(a.batch), dim3(256), 0, s, a);
  }
  return launch_status();
}

}  // namespace

LLVQ_API int64_t llvq_kv_pool_bytes(const llvq_kv_desc* d) {
  const int st = check_desc(d);
  return st != LLVQ_OK ? st : (int64_t)d->pages * d->kv_heads * block_bytes(d);
}

LLVQ_API int llvq_kv_write(const llvq_kv_desc* d, void* pool, const void* k, int64_t k_token, int64_t k_head, const void* v,
                           int64_t v_token, int64_t v_head, int32_t dtype, const llvq_batch* batch, int32_t* err_count,
                           void* stream) {
  return kv_call<true>(d, pool, k, k_token, k_head, v, v_token, v_head, dtype, batch, err_count, stream);
}

LLVQ_API int llvq_kv_read(const llvq_kv_desc* d, const void* pool, void* k, int64_t k_token, int64_t k_head, void* v,
                          int64_t v_token, int64_t v_head, int32_t dtype, const llvq_batch* batch, int32_t* err_count,
                          void* stream) {
  return kv_call<false>(d, pool, k, k_token, k_head, v, v_token, v_head, dtype, batch, err_count, stream);
}

LLVQ_API int64_t llvq_attn_workspace_bytes(const llvq_kv_desc* d, int32_t heads, int64_t tokens, int32_t batch,
                                           int32_t max_chunk, int32_t max_len) {
  int st = check_attn(d, heads, tokens, batch, max_chunk, max_len);
  if (st != LLVQ_OK) return st;
  for (const bool f32 : {false, true}) {  // either type of query
    Cut cut;
    st = cut_of(d, heads / d->kv_heads, batch, max_chunk, max_len, 0, f32, &cut);
    if (st != LLVQ_OK) return st;
  }
  // fewer sequences are split into more parts: the most that any call of no larger arguments needs
  const int64_t splits = ((int64_t)max_len + 127) / 128;
  if (splits <= 1) return 0;
  const int64_t rows = (splits < kMaxSplits ? splits : kMaxSplits) * tokens * heads, most = most_split_rows(d->head_dim);
  return workspace_of(d, rows < most ? rows : most);
}

LLVQ_API int llvq_attn(const llvq_kv_desc* d, const void* pool, const void* q, int64_t q_token, int64_t q_head, void* out,
                       int64_t out_token, int64_t out_head, int32_t dtype, int32_t heads, const llvq_batch* batch,
                       int32_t max_chunk, int32_t max_len, float scale, int32_t causal, int32_t window, void* workspace,
                       int64_t workspace_bytes, int32_t* err_count, void* stream) {
  Cache c;
  int st = make_cache(d, pool, batch, &c);
  if (st != LLVQ_OK) return st;
  st = check_attn(d, heads, batch->tokens, batch->batch, max_chunk, max_len);
  if (st != LLVQ_OK) return st;
  if (dtype != LLVQ_X_F32 && dtype != LLVQ_X_BF16) return LLVQ_EINVAL;
  const float scale_log2 = (float)((double)scale * 1.4426950408889634);
  if (!(scale > 0.0f) || !(scale_log2 < INFINITY) || window < 0 || window > kMaxLen) return LLVQ_EINVAL;
  if (err_count && !aligned(err_count, 4)) return LLVQ_EINVAL;
  if (c.tokens == 0 || c.batch == 0) return LLVQ_OK;
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
  if (cut.splits > 1) {
    a.part = static_cast<float*>(workspace);
    a.stats = a.part + (int64_t)cut.splits * c.tokens * heads * c.dim;
  }
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  const unsigned grid = (unsigned)((int64_t)c.batch * cut.row_blocks * cut.splits * c.heads);
  a.units = (int32_t)grid;
  switch (d->kind) {
    case LLVQ_KV_BF16: st = launch_attn_dp<LLVQ_KV_BF16>(a, f32, cut, grid, s); break;
    case LLVQ_KV_FP8: st = launch_attn_dp<LLVQ_KV_FP8>(a, f32, cut, grid, s); break;
    default: st = launch_attn_dp<LLVQ_KV_FP4>(a, f32, cut, grid, s); break;
  }
  if (st != LLVQ_OK || cut.splits == 1) return st;
  return f32 ? launch_join_dim<true>(a, s) : launch_join_dim<false>(a, s);
}

LLVQ_API int64_t llvq_draft_workspace_bytes(int32_t batch, int32_t vocab) {
  if (batch < 0 || batch > LLVQ_MAX_SEQS || vocab < 1) return LLVQ_EINVAL;
  // the most keys of any smaller batch too: batch * parts < 1024 + batch where a row is shared out
  const int64_t whole = batch, shared = (int64_t)batch * draft_parts(1, vocab), most = 1023 + whole;
  return 8 * (shared < most ? shared : most);
}

LLVQ_API int llvq_draft_verify(const void* target, const void* draft, int32_t dtype, const int32_t* tokens,
                               const int32_t* counts, const float* uniforms, const float* noise, int32_t batch,
                               int32_t drafts, int32_t vocab, int32_t* accepted, int32_t* out, void* workspace,
                               int64_t workspace_bytes, int32_t* err_count, void* stream) {
  if (batch < 0 || batch > LLVQ_MAX_SEQS || drafts < 0 || drafts >= kMaxDrafts || vocab < 1) return LLVQ_EINVAL;
  if (dtype != LLVQ_X_F32 && dtype != LLVQ_X_BF16) return LLVQ_EINVAL;
  if (err_count && !aligned(err_count, 4)) return LLVQ_EINVAL;
  if (batch == 0) return LLVQ_OK;
  const int size = dtype == LLVQ_X_F32 ? 4 : 2;
  if (!target || !noise || !accepted || !out || !workspace || (drafts > 0 && (!tokens || !uniforms))) return LLVQ_EINVAL;
  if (!aligned(target, size) || !aligned(draft, size) || !aligned(tokens, 4) || !aligned(counts, 4) || !aligned(uniforms, 4) ||
      !aligned(noise, 4) || !aligned(accepted, 4) || !aligned(out, 4) || !aligned(workspace, 8))
    return LLVQ_EINVAL;
  if (workspace_bytes < (int64_t)batch * draft_parts(batch, vocab) * 8) return LLVQ_EINVAL;
  DraftArgs a = {};
  a.target = target;
  a.draft = draft;
  a.tokens = tokens;
  a.counts = counts;
  a.uniforms = uniforms;
  a.noise = noise;
  a.keys = static_cast<uint64_t*>(workspace);
  a.accepted = accepted;
  a.out = out;
  a.err = err_count;
  a.batch = batch;
  a.drafts = drafts;
  a.vocab = vocab;
  a.parts = draft_parts(batch, vocab);
  a.per = (int32_t)(((int64_t)vocab + a.parts - 1) / a.parts);
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  return dtype == LLVQ_X_F32 ? launch_draft<true>(a, s) : launch_draft<false>(a, s);
}
