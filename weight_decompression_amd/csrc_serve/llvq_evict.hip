// Eviction from the paged cache: attention that gives its rows' log-sums, the attention weight that every cached token
// has received, the choice of the tokens that stay and their move to the front.
#include "attn_host.h"
#include "choose.h"
#include "keep.h"
#include "serve_host.h"
#include "weigh.h"

using namespace serve;

LLVQ_API int llvq_attn_lse(const llvq_kv_desc* d, const void* pool, const void* q, int64_t q_token, int64_t q_head, void* out,
                           int64_t out_token, int64_t out_head, int32_t dtype, int32_t heads, const llvq_batch* batch,
                           int32_t max_chunk, int32_t max_len, float scale, int32_t causal, int32_t window, float* lse,
                           void* workspace, int64_t workspace_bytes, int32_t* err_count, void* stream) {
  return attn_call<kLse>(d, pool, q, q_token, q_head, out, out_token, out_head, dtype, heads, batch, nullptr, max_chunk, max_len,
                         scale, causal, window, lse, workspace, workspace_bytes, err_count, stream);
}

namespace {

// Row tiles of 16 that the kernel for few rows takes (0: the kernel for many), waves that share out the rows of the same keys
// there, workgroups that share out a sequence's keys.
struct WeighCut {
  int tiles, team, groups;
};

inline WeighCut weigh_cut(int64_t rows, int dim, bool f32, int64_t seqs, int32_t max_len) {
  WeighCut w;
  w.team = 1;
  // Up to 32 rows the kernel for few is the faster one, with either type of queries (16 sequences of up to 16384 keys, 64 heads
  // over 8, us of one and the other: 8 rows in e4m3 49 and 97, 32 rows 51 and 83, in bf16 90 and 114, in e2m1 44 and 73; f32
  // queries, 32 rows 67 and 74, 92 and 100, 61 and 63).  Wider tiles would not leave it the registers for the loads ahead: two of
  // 256-wide f32 rows do not fit a wave.
  w.tiles = rows <= 16 ? 1 : rows <= 32 && !(f32 && dim > 128) ? 2 : 0;
  const int64_t pieces = ((int64_t)max_len + 127) / 128;  // of four waves
  if (w.tiles) {
    // up to 16 pieces a wave, fewer while that leaves places on the chip empty
    int64_t each = pieces * seqs / 1024;
    each = each < 1 ? 1 : each > 16 ? 16 : each;
    w.groups = (int)((pieces + each - 1) / each);
  } else {
    w.groups = (int)(dim <= 128 ? (pieces + 1) / 2 : pieces);
    // Where 256 keys a workgroup leave compute units idle, its waves share out the rows of 64 (2048 tokens of 32 heads over 8
    // of 128 channels in e4m3, their own keys: 64 workgroups 174 us, 256 of a quarter 73; 1024 over 4096: 128 99 us, 53; 2048 over
    // 8192: 256 177 us, 180)
    w.team = w.groups * seqs >= 256 ? 1 : !f32 ? 4 : dim <= 128 ? 2 : 1;
    w.groups *= w.team;
  }
  // (a launch has fewer than 2^32 threads)
  const int64_t most = ((1ll << 24) - 1) / seqs;
  if (w.groups > most) w.groups = (int)(most < 1 ? 1 : most);
  return w;
}

template <int KIND, int DP, int NT>
int launch_weigh_nt(const WeighArgs& a, const WeighCut& cut, hipStream_t s) {
  const dim3 grid((unsigned)a.units);
  if constexpr (NT == 1 || DP <= 128) {
    if (cut.tiles == 2) {
      hipLaunchKernelGGL((k_weigh_few<KIND, DP, NT, 2>), grid, dim3(256), 0, s, a);
      return launch_status();
    }
  }
  constexpr int kTeam = NT == 1 ? 4 : 2;
  if constexpr (NT == 1 || DP <= 128) {
    if (cut.tiles == 0 && cut.team > 1) {
      hipLaunchKernelGGL((k_weigh_many<KIND, DP, NT, kTeam>), grid, dim3(256), 0, s, a);
      return launch_status();
    }
  }
  if (cut.tiles == 1)
    hipLaunchKernelGGL((k_weigh_few<KIND, DP, NT, 1>), grid, dim3(256), 0, s, a);
  else
    hipLaunchKernelGGL((k_weigh_many<KIND, DP, NT, 1>), grid, dim3(256), 0, s, a);
  return launch_status();
}
template <int KIND, int DP>
int launch_weigh(const WeighArgs& a, bool f32, const WeighCut& cut, hipStream_t s) {
  return f32 ? launch_weigh_nt<KIND, DP, 3>(a, cut, s) : launch_weigh_nt<KIND, DP, 1>(a, cut, s);
}
template <int KIND>
int launch_weigh_dim(const WeighArgs& a, bool f32, const WeighCut& cut, hipStream_t s) {
  switch (padded_dim(a.c.dim)) {
    case 64: return launch_weigh<KIND, 64>(a, f32, cut, s);
    case 128: return launch_weigh<KIND, 128>(a, f32, cut, s);
    default: return launch_weigh<KIND, 256>(a, f32, cut, s);
  }
}

// A cache without rows of new tokens: what the choice and the move need of a batch.
int make_lists(const llvq_kv_desc* d, const void* pool, const llvq_batch* n, Cache* c) {
  if (!n || n->batch < 0 || n->batch > LLVQ_MAX_SEQS || n->max_pages < 0) return LLVQ_EINVAL;
  if (n->batch > 0 && (!n->lens || (n->max_pages > 0 && !n->table))) return LLVQ_EINVAL;
  if (!aligned(pool, 16) || !aligned(n->starts, 4) || !aligned(n->lens, 4) || !aligned(n->table, 4)) return LLVQ_EINVAL;
  const llvq_batch none = {n->starts, n->lens, n->table, n->batch, n->max_pages, 0};
  return make_cache(d, pool, &none, c);
}

}  // namespace

LLVQ_API int llvq_kv_weigh(const llvq_kv_desc* d, const void* pool, float* weights, const void* q, int64_t q_token, int64_t q_head,
                           int32_t dtype, int32_t heads, const float* lse, const llvq_batch* batch, int32_t max_chunk,
                           int32_t max_len, float scale, int32_t causal, int32_t window, int32_t fresh, int32_t* err_count,
                           void* stream) {
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
  if (!q || !lse || !weights || !aligned(q, size) || !aligned(lse, 4) || !aligned(weights, 4)) return LLVQ_EINVAL;
  if (q_token < 0 || q_head < 0) return LLVQ_EINVAL;
  if ((int64_t)max_chunk * (heads / d->kv_heads) > 0x7fffff00) return LLVQ_EINVAL;  // (row numbers, a block past the last one)
  WeighArgs a = {};
  a.c = c;
  a.q = q;
  a.lse = lse;
  a.weights = weights;
  a.q_token = q_token;
  a.q_head = q_head;
  a.share = make_divider((uint32_t)(heads / d->kv_heads));
  a.window = window;
  a.causal = causal != 0;
  a.fresh = fresh != 0;
  a.max_rows = max_chunk;
  a.q_vec = wide(q, q_token, q_head, size);
  a.scale_log2 = scale_log2;
  a.err = err_count;
  const int64_t seqs = (int64_t)c.batch * c.heads;
  if (seqs >= 1 << 24) return LLVQ_EINVAL;
  const WeighCut cut = weigh_cut((int64_t)max_chunk * a.share.by, padded_dim(d->head_dim), f32, seqs, max_len);
  a.tiles = cut.groups;
  a.units = (int32_t)(seqs * cut.groups);
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  switch (d->kind) {
    case LLVQ_KV_BF16: return launch_weigh_dim<LLVQ_KV_BF16>(a, f32, cut, s);
    case LLVQ_KV_FP8: return launch_weigh_dim<LLVQ_KV_FP8>(a, f32, cut, s);
    default: return launch_weigh_dim<LLVQ_KV_FP4>(a, f32, cut, s);
  }
}

LLVQ_API int llvq_kv_choose(const llvq_kv_desc* d, const float* weights, const llvq_batch* batch, int32_t budget, int32_t sinks,
                            int32_t recent, int32_t* keep, int32_t* counts, int32_t* err_count, void* stream) {
  Cache c;
  const int st = make_lists(d, nullptr, batch, &c);
  if (st != LLVQ_OK) return st;
  if (budget < 1 || budget > kMaxLen || sinks < 0 || recent < 0 || (int64_t)sinks + recent > budget) return LLVQ_EINVAL;
  if (err_count && !aligned(err_count, 4)) return LLVQ_EINVAL;
  if (c.batch == 0) return LLVQ_OK;
  if (!weights || !keep || !counts || !aligned(weights, 4) || !aligned(keep, 4) || !aligned(counts, 4)) return LLVQ_EINVAL;
  if ((int64_t)c.batch * c.heads * kChooseThreads >= (1ll << 32)) return LLVQ_EINVAL;
  ChooseArgs a = {};
  a.c = c;
  a.weights = weights;
  a.keep = keep;
  a.counts = counts;
  a.budget = budget;
  a.sinks = sinks;
  a.recent = recent;
  a.fours = d->page_tokens % 4 == 0 && aligned(weights, 16);
  a.err = err_count;
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  const dim3 grid((unsigned)(c.batch * c.heads));
  // By the longest sequence that the table holds: a thread holds 4 places, 32, or reads 16 at a time again for each digit.  A form
  // for more places than a sequence has costs its loads and scans (the kernel alone, 8 heads, by 4, 32 and 16 at a time: 2304
  // places 7.7, 14.0 and 19.2 us; 32768 places - , 24.0 and 39.5, of 32 sequences 32.3 and 57.4)
  const int64_t places = (int64_t)c.max_pages * c.page.by;
  if (places <= 4 * kChooseThreads)
    hipLaunchKernelGGL((k_choose<4, false>), grid, dim3(kChooseThreads), 0, s, a);
  else if (places <= 32 * kChooseThreads)
    hipLaunchKernelGGL((k_choose<32, false>), grid, dim3(kChooseThreads), 0, s, a);
  else
    hipLaunchKernelGGL((k_choose<16, true>), grid, dim3(kChooseThreads), 0, s, a);
  return launch_status();
}

LLVQ_API int llvq_kv_keep(const llvq_kv_desc* d, void* pool, float* weights, const llvq_batch* batch, const int32_t* keep,
                          int32_t lists, int32_t width, const int32_t* counts, int32_t* err_count, void* stream) {
  Cache c;
  const int st = make_lists(d, pool, batch, &c);
  if (st != LLVQ_OK) return st;
  if ((lists != 1 && lists != d->kv_heads) || width < 0 || width > kMaxLen) return LLVQ_EINVAL;
  if (!aligned(weights, 4) || !aligned(keep, 4) || !aligned(counts, 4) || (err_count && !aligned(err_count, 4))) return LLVQ_EINVAL;
  if (c.batch == 0 || width == 0) return LLVQ_OK;
  if (!pool || !keep) return LLVQ_EINVAL;
  KeepArgs a = {};
  a.c = c;
  a.weights = weights;
  a.keep = keep;
  a.counts = counts;
  a.lists = lists;
  a.width = width;
  a.from_new = batch->starts != nullptr;
  a.err = err_count;
  // A row of up to 64 bytes is a slice (four chunks at most).  Of wider ones
  // a workgroup takes whole rows of up to 256 bytes where that leaves 128 workgroups, else 128 bytes: half a line each costs
  // more than the workgroups bring (8 x 8 heads, 256 bytes: 128 us whole, 134 in halves, 161 in quarters; 4 x 8 heads 92, 66
  // and 109)
  const int64_t seqs = (int64_t)c.batch * c.heads;
  a.side = c.row <= 64 ? 4 : c.row > 128 && seqs * 2 * ((c.row + 255) / 256) >= 128 ? 16 : 8;
  a.slices = (c.row / 16 + a.side - 1) / a.side;
  a.parts = 2 * a.slices + (c.groups > 0) + (weights != nullptr);
  const int64_t grid = seqs * a.parts;
  if (grid * kKeepThreads >= (1ll << 32)) return LLVQ_EINVAL;
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  // Short lists: 256 threads leave workgroups less to wait for (the kernel alone, bf16: 16 paths of up to 6 for 8 heads 4.3 us, with
  // 1024 threads 6.3; 64 lists of 32 8.0 and 28.4); long ones need the loads of 1024 (2048 of 2304 15.5 and 11.2, 8192 of 32768 for 8
  // x 8 heads 166 and 130).  Lists of 33 to 64 would still do better with 256 (64 lists of 48 8.5 and 28.5; one of 64 4.1 and 5.7)
  hipLaunchKernelGGL(k_keep, dim3((unsigned)grid), dim3(width <= 32 ? 256 : kKeepThreads), 0, s, a);
  return launch_status();
}
