// Checks of the arguments that calls over matrices in device memory share
// (blocks.hip, groups.hip): shapes, pointers, overlaps, devices.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>
#include <initializer_list>
#include <string>

#include "reshard.h"

namespace rs {

// Keeps `msg` as the calling thread's last error and returns `s` (reshard.hip).
reshard_status_t report(reshard_status_t s, const std::string& msg);
reshard_status_t bad(const char* name, const char* what);
reshard_status_t too_many();

bool is_plain(int dtype);    // F32, BF16, F16
bool is_held(int dtype);     // FP8_E4M3, FP8_E5M2
bool is_grouped(int dtype);  // FP4_E2M1
inline bool empty(const reshard_matrix_t& m) { return m.rows == 0 || m.cols == 0; }

// Shape, type and strides of one matrix.
enum Kind { kPlain = 1, kHeld = 2, kAny = 3, kGrouped = 4 };
reshard_status_t check_shape(const reshard_matrix_t* m, const char* name, Kind kind);

// A matrix of a call, and an array of `bytes` contiguous bytes of elements of `align`.
struct Use {
  const reshard_matrix_t* m;
  const char* name;
  bool written;
};
struct Array {
  const void* data;
  int64_t bytes;
  const char* name;
  bool written;
  uint32_t align;
};

// Everything about a call's matrices and arrays that have elements, its workspace
// and the stream: what is written overlaps nothing, and all of it is memory of the
// current device.  At most kMaxUses of each.
constexpr int kMaxUses = 6;
reshard_status_t check_call(std::initializer_list<Use> uses, std::initializer_list<Array> arrays, const void* workspace,
                            int64_t need, int64_t given, void* stream);

// The status of a launch.
reshard_status_t launched(hipError_t e, const char* what);

// No exception may cross the C ABI (messages allocate).
template <typename F> reshard_status_t guarded(F call) {
  try {
    return call();
  } catch (...) {
    return RESHARD_ERR_OUT_OF_MEMORY;
  }
}

}  // namespace rs
