// Host helpers shared by the files of the C ABI: status codes with a message for
// wkv_last_error(), and the checks every entry point makes before its first HIP call.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "wkv.h"

namespace wkv {
namespace api {

// Records the message for wkv_last_error() on this thread and returns `s`.
wkv_status fail(wkv_status s, const char *fmt, ...) __attribute__((format(printf, 2, 3)));
wkv_status ok();

inline bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

inline bool dtype_ok(wkv_dtype d) { return d == WKV_F32 || d == WKV_BF16; }

inline wkv_status launched(hipError_t e, const char *what) {
  if (e != hipSuccess) return fail(WKV_ERR_DEVICE, "%s: launch failed: %s", what, hipGetErrorString(e));
  return ok();
}

constexpr int kMaxGridY = 65535;

#define REQUIRE(cond, ...)                                                  \
  do {                                                                      \
    if (!(cond)) return wkv::api::fail(WKV_ERR_INVALID_ARG, __VA_ARGS__);   \
  } while (0)

}  // namespace api
}  // namespace wkv
