// Host side of the serving calls of include/llvq.h: the paged key/value cache, the attention over it
// and the check of drafted tokens.  Arguments are validated here, before any launch; kernels bound every
// index that they read from device memory by what the host was told.
#include "attn_host.h"
#include "draft.h"
#include "kv_cache.h"
#include "serve_host.h"

using namespace serve;

namespace {

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
  return attn_call<kPlain>(d, pool, q, q_token, q_head, out, out_token, out_head, dtype, heads, batch, nullptr, max_chunk, max_len,
                           scale, causal, window, nullptr, workspace, workspace_bytes, err_count, stream);
}

LLVQ_API int64_t llvq_draft_workspace_bytes(int32_t batch, int32_t vocab) {
  if (batch < 0 || batch > LLVQ_MAX_SEQS || vocab < 1) return LLVQ_EINVAL;
  return draft_keys_bytes(batch, vocab);
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
