// Trees of drafted tokens: attention of their nodes over the paged cache (the checks and launches are those of
// llvq_attn) and the check of the trees.
#include "attn_host.h"

using namespace serve;

LLVQ_API int llvq_attn_tree(const llvq_kv_desc* d, const void* pool, const void* q, int64_t q_token, int64_t q_head, void* out,
                            int64_t out_token, int64_t out_head, int32_t dtype, int32_t heads, const llvq_batch* batch,
                            const int32_t* parents, int32_t max_chunk, int32_t max_len, float scale, int32_t window,
                            void* workspace, int64_t workspace_bytes, int32_t* err_count, void* stream) {
  return attn_call<kTree>(d, pool, q, q_token, q_head, out, out_token, out_head, dtype, heads, batch, parents, max_chunk, max_len,
                          scale, 1, window, nullptr, workspace, workspace_bytes, err_count, stream);
}
