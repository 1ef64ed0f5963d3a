// One workspace, sized once for the largest step, serves every smaller one: for drawn sizes, no call of no larger
// arguments refuses it.  Run without a device: a call that passes its checks is told that there is nothing to launch on.
// Prints "ok <checks>" and exits 0, or the sizes that failed and exits 1.

#include <hip/hip_runtime_api.h>
#include <stdint.h>
#include <stdio.h>

#include "llvq.h"

static uint64_t g_state = 12345;
static int64_t up_to(int64_t n) {  // 1..n, spread over its logarithm
  g_state = g_state * 6364136223846793005ull + 1442695040888963407ull;
  const uint64_t r = g_state >> 33;
  int64_t most = n;
  for (uint64_t half = r & 15; half && most > 1; --half) most = (most + 1) / 2;
  return 1 + (int64_t)((r >> 4) % (uint64_t)most);
}

int main() {
  int devices = 0;
  if (hipGetDeviceCount(&devices) == hipSuccess && devices > 0) {  // the pointers below are the host's
    fprintf(stderr, "a device is visible\n");
    return 1;
  }
  alignas(16) static uint8_t buf[64];
  void* p = buf;
  int32_t* ip = (int32_t*)p;
  const float* fp = (const float*)p;
  const int32_t dims[] = {32, 64, 96, 128, 160, 256};
  int checks = 0;
  for (int i = 0; i < 3000; ++i) {
    const llvq_kv_desc d = {(int32_t)up_to(3) - 1, (int32_t)up_to(32), dims[up_to(6) - 1], 16, 1 << 20};
    const int32_t heads = d.kv_heads * (int32_t)up_to(16), batch = (int32_t)up_to(256), chunk = (int32_t)up_to(4096), len = (int32_t)up_to(1 << 18);
    const int64_t tokens = up_to((int64_t)batch * chunk < (1 << 20) ? (int64_t)batch * chunk : 1 << 20);
    const int64_t size = llvq_attn_workspace_bytes(&d, heads, tokens, batch, chunk, len);
    if (size < 0) continue;
    for (int j = 0; j < 60; ++j) {
      const int32_t b = (int32_t)up_to(batch), c = (int32_t)up_to(chunk), l = (int32_t)up_to(len), w = (int32_t)(j % 3 ? 0 : up_to(len));
      const int64_t t = up_to((int64_t)b * c < tokens ? (int64_t)b * c : tokens);
      const int32_t dtype = j & 1 ? LLVQ_X_F32 : LLVQ_X_BF16;
      const llvq_batch n = {ip, ip, ip, b, 1, (int32_t)t};
      const int st = llvq_attn(&d, p, p, 1, 1, p, 4, 4, dtype, heads, &n, c, l, 0.1f, 1, w, p, size, nullptr, nullptr);
      const int64_t less = llvq_attn_workspace_bytes(&d, heads, t, b, c, l);
      ++checks;
      if (st != LLVQ_EHIP || less > size) {
        fprintf(stderr, "attn: kind %d, %d heads of %d over %d; sized for %lld tokens, %d sequences, %d, %d: %lld; refused (%d, %lld) at %lld, %d, %d, %d, window %d\n",
                d.kind, heads, d.head_dim, d.kv_heads, (long long)tokens, batch, chunk, len, (long long)size, st, (long long)less, (long long)t, b, c, l, w);
        return 1;
      }
    }
    const int32_t seqs = (int32_t)up_to(1024), vocab = (int32_t)up_to(200000);
    const int64_t bytes = llvq_draft_workspace_bytes(seqs, vocab);
    for (int j = 0; j < 20; ++j) {
      const int32_t b = (int32_t)up_to(seqs), v = (int32_t)up_to(vocab);
      ++checks;
      if (llvq_draft_verify(p, p, LLVQ_X_F32, ip, ip, fp, fp, b, 3, v, ip, ip, p, bytes, nullptr, nullptr) != LLVQ_EHIP ||
          llvq_draft_workspace_bytes(b, v) > bytes) {
        fprintf(stderr, "drafts: sized for %d x %d: %lld; refused at %d x %d\n", seqs, vocab, (long long)bytes, b, v);
        return 1;
      }
    }
  }
  printf("ok %d\n", checks);
  return 0;
}
