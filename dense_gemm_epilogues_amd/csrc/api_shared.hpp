// Shared by the files of the C ABI: the thread's last error and the check that a stream belongs to the calling
// thread's current device, which is a gfx950 (and its number of compute units), both defined in ep_api.cpp; what the
// calls without a handle check alike.
#pragma once
#include "ep.h"
#include "fp8_ops.hpp"

namespace ep {

int api_fail(int status, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
void api_clear();
int api_stream(void* stream, int* cus = nullptr);

constexpr int64_t kMaxCount = ((int64_t)1 << 31) - 4096;

inline bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }
inline ep_status done(hipError_t e, const char* what) {
  if (e != hipSuccess) return (ep_status)api_fail(EP_ERR_HIP, "%s: %s", what, hipGetErrorString(e));
  return EP_OK;
}
#define EP_REQUIRE(cond, status, ...) \
  do {                                \
    if (!(cond)) return (ep_status)api_fail(status, __VA_ARGS__); \
  } while (0)

inline ep_status check_elt(int elt) {
  EP_REQUIRE(elt == EP_ELT_F16 || elt == EP_ELT_BF16 || elt == EP_ELT_F32, EP_ERR_UNSUPPORTED, "unknown element type %d", elt);
  return EP_OK;
}

}  // namespace ep
