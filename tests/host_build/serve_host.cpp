// Host checks of the serving calls' validation and size arithmetic, built under AddressSanitizer
// and UndefinedBehaviorSanitizer (no GPU needed: every call here is refused or has nothing to do).
// Prints "ok <checks>" and exits 0, or names the first failed check and exits 1.

#include <math.h>
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
  alignas(16) static uint8_t buf[256];
  void* p = buf;
  const int32_t* ip = (const int32_t*)p;
  const llvq_kv_desc d = {LLVQ_KV_FP4, 8, 128, 16, 100};
  CHECK(llvq_kv_pool_bytes(&d) == 100ll * 8 * 2 * 16 * (64 + 4));
  const llvq_kv_desc most = {LLVQ_KV_BF16, 1024, 256, 4096, 2147483647};
  CHECK(llvq_kv_pool_bytes(&most) == 2147483647ll * 1024 * 4096 * 1024);
  const int32_t edge[] = {INT32_MIN, -1, 0, 1, 31, 33, 1025, INT32_MAX};
  for (int32_t x : edge) {
    const llvq_kv_desc a[] = {{x, 8, 128, 16, 100}, {1, x, 128, 16, 100}, {1, 8, x, 16, 100}, {1, 8, 128, x, 100}, {1, 8, 128, 16, x}};
    for (const llvq_kv_desc& e : a) {
      const int64_t n = llvq_kv_pool_bytes(&e);
      CHECK(n == LLVQ_EINVAL || n > 0);
      const int64_t w = llvq_attn_workspace_bytes(&e, 8 * 4, 100, 3, 5, 4000);
      CHECK(w == LLVQ_EINVAL || w >= 0);
      const llvq_batch none = {ip, ip, ip, 1, 1, 0};
      CHECK(llvq_kv_write(&e, p, p, 1, 1, p, 1, 1, LLVQ_X_F32, &none, nullptr, nullptr) == (n > 0 ? LLVQ_OK : LLVQ_EINVAL));
    }
    for (int32_t y : edge) {
      const int64_t w = llvq_attn_workspace_bytes(&d, 64, x, 3, y, 1 << 30);
      CHECK(w == LLVQ_EINVAL || w >= 0);
      const int64_t z = llvq_attn_workspace_bytes(&d, x, 100, y, 7, 1 << 20);
      CHECK(z == LLVQ_EINVAL || z >= 0);
      const int64_t v = llvq_draft_workspace_bytes(x, y);
      CHECK(v == LLVQ_EINVAL || v >= 0);
      const llvq_batch b = {nullptr, nullptr, nullptr, x, y, 3};
      const int st = llvq_kv_read(&d, p, p, 1, 1, p, 1, 1, LLVQ_X_F32, &b, nullptr, nullptr);
      CHECK(st == (x == 0 && y >= 0 ? LLVQ_OK : LLVQ_EINVAL));
    }
    const llvq_batch b = {ip, ip, ip, 2, 2, 3};
    CHECK(llvq_attn(&d, p, p, 1024, 128, nullptr, 1024, 128, LLVQ_X_BF16, 8, &b, x, x, 0.1f, 1, x, p, 256, nullptr, nullptr) == LLVQ_EINVAL);
    CHECK(llvq_draft_verify(p, p, LLVQ_X_F32, ip, ip, (float*)p, (float*)p, 1, x, x, nullptr, (int32_t*)p, p, 256, nullptr, nullptr) ==
          LLVQ_EINVAL);
  }
  CHECK(llvq_attn(&d, p, p, 1024, 128, p, 1024, 128, LLVQ_X_BF16, 8, nullptr, 1, 1, 0.1f, 1, 0, p, 256, nullptr, nullptr) == LLVQ_EINVAL);
  const llvq_batch nothing = {nullptr, nullptr, nullptr, 0, 0, 0};
  CHECK(llvq_attn(&d, nullptr, nullptr, 0, 0, nullptr, 0, 0, LLVQ_X_F32, 8, &nothing, 1, 1, 0.1f, 1, 0, nullptr, 0, nullptr, nullptr) ==
        LLVQ_OK);
  CHECK(llvq_attn(&d, p, p, 1, 1, p, 4, 4, LLVQ_X_F32, 8, &nothing, 1, 1, NAN, 1, 0, p, 256, nullptr, nullptr) == LLVQ_EINVAL);
  printf("ok %d\n", g_checks);
  return 0;
}
