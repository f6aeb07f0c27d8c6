// What the token-mixing kernels share with the library's entry points.
#pragma once

#include "sdv_kernels.h"

namespace sdv {

// A bit of the device status word, beside kDevErrTimeout and kDevErrTmemBase.
constexpr int kDevErrIndex = 4;  // a table entry or a length on the device out of range

// The timeout-path test hook (sdv_debug_fault): the limit of every bounded wait (0: the
// built-in one) and 1 + the stage whose copy is never issued (0: none).
struct DebugFault {
  unsigned long long wait_ns;
  int withhold;
};
DebugFault debug_fault();

}  // namespace sdv
