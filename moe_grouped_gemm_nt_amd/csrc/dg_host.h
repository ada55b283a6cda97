// Host-side helpers shared by the files that hold entry points of the C ABI:
// error reporting, alignment checks and the scratch memory of a call.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace dg {

// Sets this host thread's dg_last_error() message and returns `status`.
int fail(int status, const char* fmt, ...) __attribute__((format(printf, 2, 3)));

inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// Scratch memory of a call on a stream of the current device (the device's
// shared workspace, or the one bound to the stream), 256-byte aligned.
struct Scratch {
  int num_cus;
  uint8_t* ptr;
  size_t bytes;
};
int call_scratch(hipStream_t stream, Scratch* out);

}  // namespace dg
