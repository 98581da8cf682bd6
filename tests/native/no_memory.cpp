/* The 4-bit calls when the process has no memory left: operator new throws after a
 * countdown, for every countdown until a call no longer notices.  No exception may leave
 * a C call (it would end the process), and each answer is either the call's own refusal
 * or SBP_ENOMEM with its message.  Every call here is refused on the host: nothing is
 * launched, and the addresses are never followed. */
#include <stdint.h>
#include <stdio.h>
#include <stdlib.h>
#include <string.h>

#include <new>

#include "sbp.h"

static long g_left = -1; /* allocations until the next one fails; below 0: never */

void* operator new(size_t n) {
  if (g_left == 0) throw std::bad_alloc();
  if (g_left > 0) --g_left;
  void* p = malloc(n ? n : 1);
  if (!p) throw std::bad_alloc();
  return p;
}
void operator delete(void* p) noexcept { free(p); }
void operator delete(void* p, size_t) noexcept { free(p); }

static void* at(uintptr_t a) { return reinterpret_cast<void*>(a); }
static const void* two[2] = {reinterpret_cast<void*>(0x1000000),
                             reinterpret_cast<void*>(0x2000000)};

static int quantize(void) {  /* codes overlap x */
  return sbp_mx_quantize(at(0x1000000), SBP_BF16, 64, 96, 96, at(0x1000000), at(0x3000000),
                         nullptr, nullptr, nullptr, nullptr);
}
static int dequantize(void) {
  return sbp_mx_dequantize(at(0x2000000), at(0x3000000), 64, 96, at(0x2000000), SBP_F32, 96,
                           nullptr);
}
static int reduce(void) {
  return sbp_mx_reduce_shard(two, two, 2, 1000, nullptr, 1.0f,
                             static_cast<float*>(at(0x1000000)), nullptr);
}
static int matmul(void) {
  return sbp_mx_matmul(at(0x1000000), at(0x2000000), at(0x3000000), at(0x4000000), 300, 200, 100,
                       at(0x1000000), SBP_BF16, 200, 0, nullptr, 0, nullptr);
}
static int workspace(void) {
  return sbp_mx_matmul_workspace(1, 1, SBP_MX_MAX_K + 1) == -1 ? SBP_ERANGE : SBP_OK;
}
static int plan(void) {
  sbp_plan* p = nullptr;
  return sbp_bucket_plan(nullptr, 3, 1 << 20, 2, 8, 0, &p);
}

int main(void) {
  static const struct {
    const char* name;
    int (*call)(void);
    int status;
  } calls[] = {{"sbp_mx_quantize", quantize, SBP_EINVAL},
               {"sbp_mx_dequantize", dequantize, SBP_EINVAL},
               {"sbp_mx_reduce_shard", reduce, SBP_EINVAL},
               {"sbp_mx_matmul", matmul, SBP_EINVAL},
               {"sbp_mx_matmul_workspace", workspace, SBP_ERANGE},
               {"sbp_bucket_plan", plan, SBP_EINVAL}};
  for (const auto& c : calls) {
    int noticed = 0;
    for (long left = 0; left < 100; ++left) {
      g_left = left;
      const int status = c.call();
      const long rest = g_left;
      g_left = -1;
      char message[256];
      snprintf(message, sizeof message, "%s", sbp_last_error());
      const bool none = strstr(message, "out of host memory") != nullptr;
      if (strncmp(message, c.name, strlen(c.name)) != 0 ||
          (status != c.status && !(status == SBP_ENOMEM && none)))
        return printf("%s, %ld allocations: %d, \"%s\"\n", c.name, left, status, message), 1;
      noticed += none;
      if (rest > 0) break; /* more than the call wants */
    }
    printf("%s: out of memory %d times\n", c.name, noticed);
  }
  printf("no exception left a call\n");
  return 0;
}
