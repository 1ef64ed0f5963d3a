// Host side of the calls for drafted trees and eviction at the largest sizes they accept, built under AddressSanitizer and
// UndefinedBehaviorSanitizer and run without a device: each call passes its checks, works out its launch and is told that there
// is nothing to launch on.  Prints "ok <checks>" and exits 0, or names the first failed check and exits 1.

#include <hip/hip_runtime_api.h>
#include <stdint.h>
#include <stdio.h>

#include "llvq.h"

static int g_checks = 0;
#define CHECK(cond)                                                      \
  do {                                                                   \
    ++g_checks;                                                          \
    if (!(cond)) {                                                       \
      fprintf(stderr, "check failed at line %d: %s\n", __LINE__, #cond); \
      return 1;                                                          \
    }                                                                    \
  } while (0)

int main() {
  int devices = 0;
  if (hipGetDeviceCount(&devices) == hipSuccess && devices > 0) {  // the pointers below are the host's
    fprintf(stderr, "a device is visible\n");
    return 1;
  }
  alignas(16) static uint8_t buf[1 << 16];
  void* p = buf;
  int32_t* ip = (int32_t*)p;
  float* fp = (float*)p;
  for (int32_t vocab : {INT32_MAX, INT32_MAX - 1023, 8193, 8192, 1})
    for (int32_t batch : {1, 2, 600}) {
      const int64_t need = llvq_tree_workspace_bytes(batch, vocab);
      CHECK(need >= 8 * batch && need <= (int64_t)sizeof(buf));
      CHECK(llvq_tree_verify(p, LLVQ_X_BF16, ip, ip, ip, fp, fp, batch, LLVQ_MAX_TOKENS, vocab, LLVQ_MAX_NODES, ip, ip, ip, p, need, nullptr,
                             nullptr) == LLVQ_EHIP);
    }
  const int32_t window[] = {0, 1, 1 << 30};
  for (int32_t kind : {LLVQ_KV_BF16, LLVQ_KV_FP8, LLVQ_KV_FP4})
    for (int32_t dim : {32, 96, 256}) {
      const llvq_kv_desc d = {kind, 1024, dim, LLVQ_MAX_PAGE, INT32_MAX};
      for (int32_t w : window)
        for (int32_t dtype : {LLVQ_X_F32, LLVQ_X_BF16}) {
          const llvq_batch one = {ip, ip, ip, 1, INT32_MAX, 1};
          for (int32_t heads : {1024, 65536}) {
            const int64_t need = 1ll << 40;  // (more than any call takes)
            CHECK(llvq_attn_tree(&d, p, p, INT64_MAX / 8, INT64_MAX / 8, p, 1ll << 60, 1ll << 60, dtype, heads, &one, ip, 1, 1 << 30, 0.1f, w, p,
                                 need, nullptr, nullptr) == LLVQ_EHIP);
            CHECK(llvq_attn_lse(&d, p, p, INT64_MAX / 8, INT64_MAX / 8, p, 1ll << 60, 1ll << 60, dtype, heads, &one, 1, 1 << 30, 0.1f, 1, w, fp, p,
                                need, nullptr, nullptr) == LLVQ_EHIP);
            CHECK(llvq_kv_weigh(&d, p, fp, p, INT64_MAX / 8, INT64_MAX / 8, dtype, heads, fp, &one, 1, 1 << 30, 0.1f, 1, w, 1, nullptr, nullptr) ==
                  LLVQ_EHIP);
          }
          // the most rows and tokens, and the most sequences that a launch of the weights takes
          const llvq_batch rows = {ip, ip, ip, 1, INT32_MAX, 32767};
          CHECK(llvq_kv_weigh(&d, p, fp, p, 1, 1, dtype, 65536, fp, &rows, 32767, 1 << 30, 0.1f, 1, w, 0, nullptr, nullptr) == LLVQ_EHIP);
          const llvq_batch seqs = {ip, ip, ip, (1 << 14) - 1, INT32_MAX, 1 << 14};
          CHECK(llvq_kv_weigh(&d, p, fp, p, 1, 1, dtype, 1024, fp, &seqs, 1 << 16, 1 << 30, 0.1f, 1, w, 0, nullptr, nullptr) == LLVQ_EHIP);
        }
      const llvq_batch all = {ip, ip, ip, (1 << 12) - 1, INT32_MAX, INT32_MAX};
      CHECK(llvq_kv_choose(&d, fp, &all, 1 << 30, 1 << 29, 1 << 29, ip, ip, nullptr, nullptr) == LLVQ_EHIP);
      const int32_t most = ((1 << 22) - 1) / (1024 * (dim / 32 + 4));
      const llvq_batch moved = {ip, ip, ip, most, INT32_MAX, INT32_MAX};
      CHECK(llvq_kv_keep(&d, p, fp, &moved, ip, 1024, 1 << 30, ip, nullptr, nullptr) == LLVQ_EHIP);
      CHECK(llvq_kv_keep(&d, p, nullptr, &moved, ip, 1, 1, nullptr, nullptr, nullptr) == LLVQ_EHIP);
    }
  printf("ok %d\n", g_checks);
  return 0;
}
