// Host side of the serving calls at the largest sizes they accept, built under AddressSanitizer and
// UndefinedBehaviorSanitizer and run without a device: each call passes its checks, works out its launch and is
// told that there is nothing to launch on.  Prints "ok <checks>" and exits 0, or names the first failed check and exits 1.

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
  const float* fp = (const float*)p;
  for (int32_t vocab : {INT32_MAX, INT32_MAX - 1023, INT32_MAX - 1024, 8193, 8192, 1})
    for (int32_t batch : {1, 2, 600}) {
      const int64_t need = llvq_draft_workspace_bytes(batch, vocab);
      CHECK(need >= 8 * batch && need <= (int64_t)sizeof(buf));
      CHECK(llvq_draft_verify(p, p, LLVQ_X_BF16, ip, nullptr, fp, fp, batch, LLVQ_MAX_DRAFTS, vocab, ip, ip, p, need, nullptr, nullptr) ==
            LLVQ_EHIP);
    }
  // keys: the longest lengths and windows, the largest pages, the most heads
  const int32_t window[] = {0, 1, 1 << 30};
  for (int32_t kind : {LLVQ_KV_BF16, LLVQ_KV_FP8, LLVQ_KV_FP4})
    for (int32_t dim : {32, 96, 256})
      for (int32_t w : window)
        for (int32_t dtype : {LLVQ_X_F32, LLVQ_X_BF16}) {
          const llvq_kv_desc d = {kind, 1024, dim, LLVQ_MAX_PAGE, INT32_MAX};
          const llvq_batch one = {ip, ip, ip, 1, INT32_MAX, 1};
          const int64_t need = llvq_attn_workspace_bytes(&d, 65536, 1, 1, 1, 1 << 30);
          CHECK(need >= 0);
          CHECK(llvq_attn(&d, p, p, INT64_MAX / 8, INT64_MAX / 8, p, 1ll << 60, 1ll << 60, dtype, 65536, &one, 1, 1 << 30, 0.1f, 1, w, p, need,
                          nullptr, nullptr) == LLVQ_EHIP);
          CHECK(llvq_kv_write(&d, p, p, 1, 1, p, 1, 1, dtype, &one, nullptr, nullptr) == LLVQ_EHIP);
          const llvq_batch all = {ip, ip, ip, LLVQ_MAX_SEQS, INT32_MAX, LLVQ_MAX_TOKENS};
          CHECK(llvq_kv_read(&d, p, p, 1, 1, p, 1, 1, dtype, &all, nullptr, nullptr) == LLVQ_EHIP);
        }
  printf("ok %d\n", g_checks);
  return 0;
}
