// Eviction from the paged cache: attention that gives its rows' log-sums, the attention weight that every cached token
// has received, the choice of the tokens that stay and their move to the front.
#include "attn_host.h"

using namespace serve;

LLVQ_API int llvq_attn_lse(const llvq_kv_desc* d, const void* pool, const void* q, int64_t q_token, int64_t q_head, void* out,
                           int64_t out_token, int64_t out_head, int32_t dtype, int32_t heads, const llvq_batch* batch,
                           int32_t max_chunk, int32_t max_len, float scale, int32_t causal, int32_t window, float* lse,
                           void* workspace, int64_t workspace_bytes, int32_t* err_count, void* stream) {
  return attn_call<kLse>(d, pool, q, q_token, q_head, out, out_token, out_head, dtype, heads, batch, nullptr, max_chunk, max_len,
                         scale, causal, window, lse, workspace, workspace_bytes, err_count, stream);
}
