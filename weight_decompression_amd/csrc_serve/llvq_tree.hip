// Trees of drafted tokens: attention of their nodes over the paged cache (the checks and launches are those of
// llvq_attn) and the check of the trees.
#include "attn_host.h"
#include "serve_host.h"
#include "tree.h"

using namespace serve;

LLVQ_API int llvq_attn_tree(const llvq_kv_desc* d, const void* pool, const void* q, int64_t q_token, int64_t q_head, void* out,
                            int64_t out_token, int64_t out_head, int32_t dtype, int32_t heads, const llvq_batch* batch,
                            const int32_t* parents, int32_t max_chunk, int32_t max_len, float scale, int32_t window,
                            void* workspace, int64_t workspace_bytes, int32_t* err_count, void* stream) {
  return attn_call<kTree>(d, pool, q, q_token, q_head, out, out_token, out_head, dtype, heads, batch, parents, max_chunk, max_len,
                          scale, 1, window, nullptr, workspace, workspace_bytes, err_count, stream);
}

namespace {

template <bool F32>
int launch_tree(const TreeArgs& a, hipStream_t s) {
  if (a.parts == 1) {
    hipLaunchKernelGGL((k_tree_one<F32>), dim3(a.batch), dim3(1024), 0, s, a);
  } else {
    hipLaunchKernelGGL((k_tree_part<F32>), dim3(a.parts, a.batch), dim3(256), 0, s, a);
    hipLaunchKernelGGL((k_tree_pick<F32>), dim3(a.batch), dim3(256), 0, s, a);
  }
  return launch_status();
}

}  // namespace

LLVQ_API int64_t llvq_tree_workspace_bytes(int32_t batch, int32_t vocab) {
  if (batch < 0 || batch > LLVQ_MAX_SEQS || vocab < 1) return LLVQ_EINVAL;
  return draft_keys_bytes(batch, vocab);
}

LLVQ_API int llvq_tree_verify(const void* target, int32_t dtype, const int32_t* starts, const int32_t* tokens,
                              const int32_t* parents, const float* uniforms, const float* noise, int32_t batch, int32_t nodes,
                              int32_t vocab, int32_t width, int32_t* accepted, int32_t* path, int32_t* out, void* workspace,
                              int64_t workspace_bytes, int32_t* err_count, void* stream) {
  if (batch < 0 || batch > LLVQ_MAX_SEQS || nodes < 0 || nodes > LLVQ_MAX_TOKENS || vocab < 1) return LLVQ_EINVAL;
  if (width < 1 || width > LLVQ_MAX_NODES || (dtype != LLVQ_X_F32 && dtype != LLVQ_X_BF16)) return LLVQ_EINVAL;
  if (err_count && !aligned(err_count, 4)) return LLVQ_EINVAL;
  if (batch == 0) return LLVQ_OK;
  if (!starts || !noise || !accepted || !path || !out || !workspace) return LLVQ_EINVAL;
  if (nodes > 0 && (!target || !tokens || !parents || !uniforms)) return LLVQ_EINVAL;
  if (!aligned(target, dtype == LLVQ_X_F32 ? 4 : 2) || !aligned(starts, 4) || !aligned(tokens, 4) || !aligned(parents, 4) ||
      !aligned(uniforms, 4) || !aligned(noise, 4) || !aligned(accepted, 4) || !aligned(path, 4) || !aligned(out, 4) ||
      !aligned(workspace, 8))
    return LLVQ_EINVAL;
  if (workspace_bytes < (int64_t)batch * draft_parts(batch, vocab) * 8) return LLVQ_EINVAL;
  TreeArgs a = {};
  a.target = target;
  a.starts = starts;
  a.tokens = tokens;
  a.parents = parents;
  a.uniforms = uniforms;
  a.noise = noise;
  a.keys = static_cast<uint64_t*>(workspace);
  a.accepted = accepted;
  a.path = path;
  a.out = out;
  a.err = err_count;
  a.batch = batch;
  a.nodes = nodes;
  a.vocab = vocab;
  a.width = width;
  a.parts = draft_parts(batch, vocab);
  a.per = (int32_t)(((int64_t)vocab + a.parts - 1) / a.parts);
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  return dtype == LLVQ_X_F32 ? launch_tree<true>(a, s) : launch_tree<false>(a, s);
}
