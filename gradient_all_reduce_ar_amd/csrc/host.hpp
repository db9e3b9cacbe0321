// host.hpp -- what the files of the C ABI share: the thread's error state,
// enum arguments as integers, and a plan's small host-side device objects.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>
#include <cstring>
#include <string>
#include <vector>

#include "../../include/ar.h"

namespace ar_host {

// Records the calling thread's error (ar_last_error, ar_last_status).
ar_status_t fail(ar_status_t st, const std::string &msg);
ar_status_t hip_fail(hipError_t e, const char *what);

// The value of a C enum argument as an integer, read from its bytes: a
// caller may pass any int, and loading a value outside the enumerators as
// the C++ enum type is undefined behaviour.
template <class E>
int32_t raw_enum(const E &v) {
  static_assert(sizeof(E) == sizeof(int32_t), "C enums are int-sized");
  int32_t r;
  std::memcpy(&r, &v, sizeof r);
  return r;
}

// The calls in flight of one plan: per stream it has run on, an event that
// the last kernel of each call records by its own dispatch (none while the
// caller captures the stream).
class CallMarks {
 public:
  // The event for a call on s; *ev = nullptr while s is being captured.
  ar_status_t of(hipStream_t s, hipEvent_t *ev);
  void wait() const;
  void release();  // waits, then drops the events

 private:
  static constexpr size_t kMax = 16;
  struct Mark {
    hipStream_t stream;
    hipEvent_t event;
  };
  std::vector<Mark> marks_;
};

// Copies `bytes` to the current device's memory on a non-blocking stream of
// its own, which it waits for.
hipError_t upload(void *dst, const void *src, size_t bytes);
// Allocates `bytes` on the current device and fills them from src, if not NULL.
hipError_t device_table(void **dst, const void *src, size_t bytes);
// AR_ERR_INVALID_ARG while the caller captures s: a plan cannot be prepared then.
ar_status_t refuse_capture(hipStream_t s);

}  // namespace ar_host
