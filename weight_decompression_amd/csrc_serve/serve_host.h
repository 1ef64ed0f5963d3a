// Host side that the units of the serving calls share: checks of the descriptors and batches of include/llvq.h.
#pragma once

#include "llvq.h"
#include "serve_common.h"

#define LLVQ_API extern "C" __attribute__((visibility("default")))

namespace serve {
namespace {

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
inline int launch_status() { return hipGetLastError() == hipSuccess ? LLVQ_OK : LLVQ_EHIP; }

inline int64_t block_bytes(const llvq_kv_desc* d) {
  const int64_t groups = d->kind == LLVQ_KV_BF16 ? 0 : d->head_dim / kGroup;
  return (2 * d->page_tokens * (code_bytes(d->kind, d->head_dim) + groups) + 15) / 16 * 16;
}

inline int check_desc(const llvq_kv_desc* d) {
  if (!d || d->kind < LLVQ_KV_BF16 || d->kind > LLVQ_KV_FP4) return LLVQ_EINVAL;
  if (d->kv_heads < 1 || d->kv_heads > 1024 || d->pages < 1) return LLVQ_EINVAL;
  if (d->head_dim < kGroup || d->head_dim > LLVQ_MAX_HEAD_DIM || d->head_dim % kGroup) return LLVQ_EINVAL;
  if (d->page_tokens < 1 || d->page_tokens > LLVQ_MAX_PAGE) return LLVQ_EINVAL;
  return LLVQ_OK;
}

inline int make_cache(const llvq_kv_desc* d, const void* pool, const llvq_batch* n, Cache* c) {
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
inline bool wide(const void* p, int64_t token, int64_t head, int bytes) {
  return aligned(p, 16) && (token * bytes) % 16 == 0 && (head * bytes) % 16 == 0;
}

}  // namespace
}  // namespace serve
